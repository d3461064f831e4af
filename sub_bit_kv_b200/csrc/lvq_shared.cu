// Decode attention for groups of requests that share coded prefixes.
//
// "LoopVQ summary", section "premises and limits": the attention reads only the step-t slice of
// each codebook, splits the coded tokens and merges the splits, and the bf16 sink and recent
// tokens, by logsumexp; section "how it differs": RoPE is applied to the reconstructed key.  Here
// the coded tokens that a group's requests have in common are restored and rotated once, and
// scored against every query of the group.
//
// Work.  A KV head's work is a list of entries: for every group its shared tokens, once per tile of
// 16 query rows (request, query head of the KV head); then for every request its own tokens (the
// rest of its coded ones, sink and recent window), once per 8 of its query heads.  An entry costs
// its 16-token tiles and a fixed overhead per query tile; the list is cut into k parts of equal
// cost, and CTA (j, h) takes part j of KV head h.  Every CTA derives the same cut from the
// counters.  All 8 warps of a CTA work on one shared entry at a time; the own entries of a part
// are cut once more, a contiguous run of tiles to a warp, so that the latencies of 8 small entries
// overlap.  Per entry it covers, a CTA leaves one partial (m, l, o) per query row; every row has a
// slot per part and kind (shared, own), and the merge kernel joins the ones that are not empty.
// Every sum is taken in a fixed order.
#include <cuda_fp16.h>

#include "lvq_common.cuh"

namespace lvq {

namespace {

constexpr int kQT = 16;                 // query rows of a tile of shared tokens
constexpr int kOT = 8;                  // query heads of a tile of own tokens
constexpr int kTT = 16;                 // tokens of a tile: two pages
// Costs in token tiles: a query tile of a shared entry as such (fragments, joining the warps), one of an own entry, and
// what the first part with own entries spends on getting to them; and what a tile of own tokens weighs against a
// shared one (its bytes are new to L2, and its warps wait for more of them).  Swept one after the other over 64 shapes
// whose inputs L2 does not hold to their least geometric mean: 32.1 us (32.5 with both tiles alike and a stage of 20).
constexpr int kSharedCost = 8, kOwnCost = 4, kOwnStage = 40;
constexpr int kSharedWeight = 8, kOwnWeight = 9;
constexpr int kWarps = 8;
constexpr int kShThreads = 32 * kWarps;
constexpr float kNoMax = -3.40282347e38f;   // softmax reference before the first token: the lowest float, which no score is below

struct SharedArgs {
  int layer, step, batch, ng, k;
  const __nv_bfloat16* q;
  const int32_t *ctx_len, *coded_len, *gb, *gt;
  const __nv_bfloat16 *sink, *ring;
  const uint8_t* idx;
  const __nv_bfloat16* cbp;
  const float* rope;
  float* po;                            // partial outputs [B][Hq][max_splits][2][d]
  float2* pml;                          // their (m, l), log2 domain
  int32_t* st;
};

// Counters of the batch in shared memory, and the partition's running costs.
struct Counters {
  long long *gcum, *ocum;               // [ng + 1], [batch + 1]: cost of the shared (own) entries before each
  int *ctx, *coded, *own0;              // [batch]: context (0: unusable), coded tokens, shared tokens of its group
  int *gb, *sh, *lead;                  // [ng + 1], [ng], [ng]: first request, shared tokens, first usable request
};
constexpr int counter_bytes(int batch, int ng) { return 8 * (ng + batch + 2) + 4 * (3 * batch + 3 * ng + 1); }

__device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }
// a / b of non-negative costs: a 64-bit division takes some hundred instructions, and only absurd batches need one
__device__ inline long long div_cost(long long a, long long b) {
  return (unsigned long long)(a | b) >> 32 ? a / b : (long long)((unsigned)a / (unsigned)b);
}

// Token tiles, query tiles and fixed cost of a query tile.
struct Entry {
  int tiles, qtiles, fixed;
  int coded, weight;                    // own entries: tiles [0, coded) are coded, the others cost `weight` each
  __device__ int units() const { return coded + (tiles - coded) * weight; }
  __device__ int tile_at(int u) const { return u <= coded ? u : coded + ceil_div(u - coded, weight); }   // first one at or past unit u
  __device__ long long each() const { return fixed + units(); }
  __device__ long long cost() const { return tiles ? qtiles * each() : 0; }
};
__device__ inline Entry shared_entry(const Geo& g, const Counters& c, int i) {
  const int tiles = ceil_div(c.sh[i], kTT);
  return {tiles, ceil_div((c.gb[i + 1] - c.gb[i]) * (g.Hq / g.H), kQT), kSharedCost, tiles, 1};
}
__device__ inline Entry own_entry(const Geo& g, const Counters& c, int b) {
  const int rep = g.Hq / g.H, coded = ceil_div(c.coded[b] - c.own0[b], kTT);
  // (a bf16 tile takes a warp 3100 cycles with one query head, like a coded one, and about a third more for each further)
  return {coded + ceil_div(c.ctx[b] - c.coded[b], kTT), ceil_div(rep, kOT), kOwnCost, coded, (min(rep, kOT) + 2) / 3};
}

// The entry of [0, n) in which cost x lies, n if x is not below the total.
__device__ inline int locate(const long long* cum, int n, long long x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (cum[mid + 1] > x) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// cum[i + 1] = the sum of the threads' costs 0 .. i, of both lists (thread i: entry i of each).  `part`: two values a
// warp.
__device__ inline void scan_costs(long long (&up)[2], const Counters& c, int ng, int batch, long long* part) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long v = __shfl_up_sync(0xffffffffu, up[k], o);
      if (lane >= o) up[k] += v;
    }
  if (lane == 31) { part[2 * warp] = up[0]; part[2 * warp + 1] = up[1]; }
  __syncthreads();
  for (int w = 0; w < warp; ++w) { up[0] += part[2 * w]; up[1] += part[2 * w + 1]; }
  if (tid < ng) c.gcum[tid + 1] = up[0];
  if (tid < batch) c.ocum[tid + 1] = up[1];
  if (tid == 0) c.gcum[0] = c.ocum[0] = 0;
  __syncthreads();
}

// Loads and checks the counters and derives the costs, a thread to a request and to a group; returns false (for
// every thread) if group_begin is not as described.
__device__ bool load_counters(const Geo& g, const SharedArgs& a, Counters& c, long long* part, bool report) {
  static_assert(kSharedMaxBatch <= kShThreads, "a thread to a request");
  const int t = threadIdx.x;
  bool ok = true;
  int ctx = 0, L = 0, v = 0, next = 0, tokens = 0;
  if (t < a.batch) { ctx = __ldcg(a.ctx_len + t); L = __ldcg(a.coded_len + t); }
  if (t < a.ng) { v = __ldcg(a.gb + t); next = __ldcg(a.gb + t + 1); tokens = __ldcg(a.gt + t); }
  if (t < a.ng) {
    ok = v >= 0 && next >= v && next <= a.batch && (t > 0 || v == 0) && (t < a.ng - 1 || next == a.batch);
    c.gb[t] = v;
    if (t == a.ng - 1) c.gb[a.ng] = next;
    c.sh[t] = max(0, tokens) / kPage * kPage;
    c.lead[t] = a.batch;
  }
  if (t < a.batch) {
    const int recent = ctx - min(g.S, max(ctx, 0)) - L;
    const bool bad = ctx < 1 || ctx > g.max_ctx || L < 0 || L > g.P * kPage || (L > 0 && ctx < g.S + L) || recent < 0 || recent > g.R;
    if (bad) {
      if (report) set_status(a.st, LVQ_ECAPACITY);
      ctx = L = 0;
    }
    c.ctx[t] = ctx;
    c.coded[t] = L;
  }
  if (__syncthreads_or(!ok)) {
    if (t == 0 && report) set_status(a.st, LVQ_EINVAL);
    return false;
  }
  // a group shares no more than its shortest usable request has coded
  int grp = 0;
  if (t < a.batch) {
    int hi = a.ng;                               // the last group that begins at or before the request
    while (hi - grp > 1) {
      const int mid = (grp + hi) / 2;
      if (c.gb[mid] <= t) grp = mid; else hi = mid;
    }
    if (ctx > 0) {
      atomicMin(&c.sh[grp], L / kPage * kPage);
      atomicMin(&c.lead[grp], t);
    }
  }
  __syncthreads();
  if (t < a.ng && c.lead[t] == a.batch) c.sh[t] = 0;   // no usable request
  if (t < a.batch) c.own0[t] = ctx > 0 ? c.sh[grp] : 0;
  long long cost[2] = {t < a.ng ? shared_entry(g, c, t).cost() : 0, t < a.batch ? own_entry(g, c, t).cost() : 0};
  scan_costs(cost, c, a.ng, a.batch, part);
  return true;
}

// Pool mode: the rows of a group name the same pages for its shared tokens.  The CTAs share the comparison (an int
// counts a CTA's: calls that need more are refused).
__device__ void check_rows(const Geo& g, const SharedArgs& a, const Counters& c) {
  const int n_cta = gridDim.x * gridDim.y, me = blockIdx.y * gridDim.x + blockIdx.x;
  bool differ = false;
  for (int e = 0; e < a.ng; ++e) {
    const int pages = c.sh[e] / kPage, first = c.lead[e], others = c.gb[e + 1] - first - 1;
    if (pages == 0 || others < 1) continue;
    // this CTA's pages of the group's list, against the rows of all its other requests
    const int p0 = (int)((long long)pages * me / n_cta), n = (int)((long long)pages * (me + 1) / n_cta) - p0;
    const int32_t* lead_row = g.pt + (size_t)first * g.pts + p0;
    const int total = n * others;
#pragma unroll 4
    for (int i = threadIdx.x; i < total; i += kShThreads) {
      const int b = first + 1 + i / n, p = i % n;
      if (c.ctx[b] > 0) differ |= __ldcg(lead_row + p) != __ldcg(g.pt + (size_t)b * g.pts + p0 + p);
    }
  }
  if (differ) set_status(a.st, LVQ_EINVAL);
}

// A query tile of an entry: rows r < nrows are (request, query head) pairs.
struct RowTile {
  int b0, rep, r0, nrows, h;
  __device__ int request(int r) const { return b0 + (r0 + r) / rep; }
  __device__ int head(int r) const { return h * rep + (r0 + r) % rep; }
};

template <int D, int C>
struct Sh {
  static constexpr int F = D / 2;                  // RoPE frequencies
  static constexpr int NG = D / C, NP = NG / 2;    // groups, pair-groups (groups P, P + NP)
  static constexpr int NI = NP / 4;                // pair-groups of a lane: P = quad + 4 i
  static constexpr int NW = D / 16;                // frequency pairs of a lane; k16 steps of a score
  static constexpr int NT = D / 8;                 // n8 tiles of an output row
  // Shared entries of 8 channels or more: a tile's second page is scored against queries turned 8 positions back, so
  // that a key's rotation moves on once a tile (32 behind 32K at c = 8: 152 us against 159; at c = 4, where the
  // loads of smaller entries leave the loop less to save, 79 against 74)
  static constexpr bool BACK = C >= 8;
  static constexpr int PAGE = NG * kPage;          // bytes of one K (or V) page
  static constexpr int STAGE = 4 * PAGE;           // a tile's codes: K pages, V pages
  static constexpr int KS = kEntries * D * 2;      // a step slice
  static constexpr int VROW = D * 2 + 16;          // a padded row of the value slice
  static constexpr int OROW = D + 4;               // a padded row of a warp's output, in floats
  // a warp's area: code stages, a query tile's fragments or 8 output rows, then 8 output rows parked
  // (a shared entry's 16 output rows take both; before them, the parked rows' place of area w holds k step w of the
  // queries turned back)
  static constexpr int WARP = kQT * OROW * 4;
  static constexpr int PARK = kOT * OROW * 4;
  static constexpr int NST = PARK / STAGE < 6 ? PARK / STAGE : 6;
  static constexpr int OFF_V = KS;
  static constexpr int OFF_W = OFF_V + (kEntries * VROW + 15) / 16 * 16;
  static constexpr int OFF_Q = OFF_W + kWarps * WARP;
  static constexpr int OFF_F = OFF_Q + 2 * NW * 32 * 16;
  static constexpr int OFF_E = OFF_F + NW * 32 * 16;
  static constexpr int OFF_R = OFF_E + 2 * NW * 4 * 16;
  static constexpr int OFF_ML = OFF_R + kWarps * F * 8;
  static constexpr int OFF_INV = OFF_ML + kWarps * kQT * 8;
  static constexpr int OFF_RED = OFF_INV + kQT * 4;
  static constexpr int OFF_BAR = OFF_RED + 4 * kWarps * 4;
  static constexpr int OFF_P = OFF_BAR + 16;
  static constexpr int OFF_C = OFF_P + 2 * kWarps * 8;
  static constexpr int smem(int batch, int ng) { return OFF_C + counter_bytes(batch, ng); }
  static_assert(NP % 4 == 0 && NI * C == 2 * NW, "lane mapping");
  static_assert(NST >= 3 && NST <= 8, "stages (a tile's RoPE row is read before the one 8 tiles on is fetched)");
  static_assert(PARK >= NW * 32 * 16 && WARP - PARK >= 2 * 32 * 16 && NW <= kWarps, "the warps' areas");
  static_assert(OFF_C + counter_bytes(kSharedMaxBatch, kSharedMaxBatch) <= 227 * 1024, "shared memory");
  static_assert(OFF_W % 16 == 0 && PARK % 16 == 0 && OFF_F % 16 == 0 && OFF_BAR % 8 == 0 && OFF_C % 8 == 0, "alignment");
};

__device__ inline uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// v minus the fp16 pair h, with one mixed-precision fused multiply-add each
__device__ inline float2 minus_h2(float2 v, uint32_t h) {
  float2 r;
  asm("{\n .reg .b16 a, b, m;\n mov.b32 {a, b}, %4;\n mov.b16 m, 0xBC00;\n fma.rn.f32.f16 %0, a, m, %2;\n"
      " fma.rn.f32.f16 %1, b, m, %3;\n}\n"
      : "=f"(r.x), "=f"(r.y) : "f"(v.x), "f"(v.y), "r"(h));
  return r;
}
// a pair of values as the sum of two fp16 pairs: hi + lo, good to 2^-22 of each value (2^-25 at least)
__device__ inline void split_h2(float2 v, uint32_t& hi, uint32_t& lo) {
  hi = pack_h2(v.x, v.y);
  const float2 r = minus_h2(v, hi);
  lo = pack_h2(r.x, r.y);
}
__device__ inline float2 b2_lohi(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }

__device__ inline void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ inline void ldmatrix4_trans(uint32_t (&v)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr) : "memory");
}
__device__ inline float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ inline void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
__device__ inline void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ inline void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }
__device__ inline void prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" :: "l"(src), "r"(bytes) : "memory");
}
__device__ inline void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ inline void dependents_may_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// 2^e as a float, e clamped to the normal range
__device__ inline float pow2i(int e) { return __int_as_float((min(max(e, -126), 127) + 127) << 23); }
// the power of two that brings magnitudes up to that bf16 below 2^14 (none where all are zero; its reciprocal
// and its products with weights up to 2^14 stay normal floats)
__device__ inline int fit_exp(uint32_t bits) { return bits ? min(13 - ((int)(bits >> 7) - 127), 90) : 0; }
__device__ inline int fit_exp_f(float m) { return m > 0.f && m < INFINITY ? min(13 - (((__float_as_int(m) >> 23) & 255) - 127), 90) : 0; }

// Channel of output tile i, fragment column n: the order in which the value fragments are restored.
template <int D, int C>
__device__ inline int out_channel(int i, int n) { return C == 4 ? n * (D / 8) + i : 8 * i + n; }

// A warp's running softmax over its tokens: m is a reference no more than 2^14 below the largest weight,
// p = 2^(s - m).  Shared entries: lane (r, quad) holds rows r and r + 8.  Own entries (stacked): rows 0-7
// are the query heads with the operands' high parts, rows 8-15 the same with the low ones, so lane (r, quad)
// holds both halves of row r, and only m[0], l[0] are used.
template <int D, int C>
struct State {
  float o[Sh<D, C>::NT][4];
  float m[2], l[2];
  __device__ void clear() {
#pragma unroll
    for (int i = 0; i < Sh<D, C>::NT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
    m[0] = m[1] = kNoMax;
    l[0] = l[1] = 0.f;
  }
};

// What the restoration of coded tokens needs, per CTA and lane.
template <int D, int C>
struct Book {
  const unsigned char *Ks, *Vs;         // step slices: keys bf16, values scaled fp16 in padded rows
  const float4* Ff;                     // [frequency pair][lane]: (cos, cos, sin, sin) at (S % 8 + j)
  const float4* E8;                     // [frequency pair][quad]: e^{i 8 theta}, (cos, cos, sin, sin); then e^{i 16 theta}
  float ks, kinv;                       // key scale (a power of two) and its reciprocal
};

// A run of coded tokens of one request (or of a group's first): logical pages [pg0, pg_end), n tokens.
struct Run {
  int lead, pg0, pg_end, n;
  const uint8_t *kcode, *vcode;         // code streams (pool mode: pools) of the head
  int ids, ids_at;                      // physical pages [ids_at, ids_at + 32) of the run, one a lane
};

// Tile t's codes into its stage; every eighth tile's RoPE row (of its first page) as well.
template <int D, int C>
__device__ __forceinline__ void fetch_tile(const Geo& g, const SharedArgs& a, Run& run, int t, unsigned char* stages, float4* rrow) {
  using X = Sh<D, C>;
  const int lane = threadIdx.x & 31, pp = 2 * t;
  if (pp - run.ids_at >= 32) {
    run.ids_at = pp;
    run.ids = phys_page(g, run.lead, min(run.pg0 + pp + lane, run.pg_end - 1));
    if (run.ids < 0) {
      set_status(a.st, LVQ_ECAPACITY);
      run.ids = 0;
    }
  }
  const int i0 = __shfl_sync(0xffffffffu, run.ids, pp - run.ids_at), i1 = __shfl_sync(0xffffffffu, run.ids, pp + 1 - run.ids_at);
  const uint32_t dst = smem_addr(stages) + (t % X::NST) * X::STAGE;
  constexpr int VP = X::PAGE / 16;
#pragma unroll
  for (int v = lane; v < 4 * VP; v += 32) {
    const int id = (v / VP) & 1 ? i1 : i0;
    cp_async16(dst + v * 16, (v < 2 * VP ? run.kcode : run.vcode) + (size_t)id * X::PAGE + v % VP * 16);
  }
  if (t % 8 == 0 && lane < X::F / 2)
    cp_async16(smem_addr(rrow) + lane * 16,
               reinterpret_cast<const float4*>(a.rope) + (size_t)(run.pg0 + pp + (g.S >> 3)) * (X::F / 2) + lane);
}
// The first tiles of a run are on their way: called as early as the pages are known, and once before coded_run.
template <int D, int C>
__device__ __forceinline__ void begin_run(const Geo& g, const SharedArgs& a, Run& run, unsigned char* stages, float4* rrow) {
#pragma unroll
  for (int t = 0; t < Sh<D, C>::NST - 1; ++t) {
    if (t * kTT < run.n) fetch_tile<D, C>(g, a, run, t, stages, rrow);
    cp_commit();
  }
}

// o += weights x values of a tile.  The tensor core cuts its sums off towards zero, so a tile's product starts from
// zero and is added in fp32, rounded to nearest: carried through a run's products the cut biases an output by
// 1.4e-6 of its size after 60 of them (measured), this way it is lost in the rounding.
template <bool STK>
__device__ inline void add_values(float (&o)[4], const uint32_t (&ph)[4], const uint32_t (&pl)[4], uint32_t b0, uint32_t b1) {
  float t[4] = {0.f, 0.f, 0.f, 0.f};
  if constexpr (!STK) mma_f16(t, pl, b0, b1);
  mma_f16(t, ph, b0, b1);
#pragma unroll
  for (int k = 0; k < 4; k += 2) {
    const float2 r = __fadd2_rn(make_float2(o[k], o[k + 1]), make_float2(t[k], t[k + 1]));
    o[k] = r.x;
    o[k + 1] = r.y;
  }
}

// Restores the run's tokens tile by tile and adds them to the state.  STK: stacked rows.  Per tile, lane
// (j, quad) restores token j of each of the two pages: the entries of pair-groups P = quad + 4 i straight
// into the B fragments of mma.sync m16n8k16 (the order of a dot product's channels is free, so a fragment's k
// indices are the channels of the lane's own entries), rotated in fp32 by e^{i p theta}, which moves on by a
// page (8 positions; Sh::BACK: by two) with one complex multiplication and is taken anew from the tables every
// 16 pages.  Keys and queries enter as sums of two fp16 values, good to 2^-22 of the largest; lo x lo is left
// out of 16 rows.  Weights too are sums of two fp16 values; values are exact.
// Query fragments: qf in registers (stacked rows), or qs in shared memory, [hi, lo][k step] 32 lanes apart
// (qs1: turned back for a tile's second page, [k step][hi, lo]).
template <int D, int C, bool STK>
__device__ __forceinline__ void coded_run(const Geo& g, const SharedArgs& a, const Book<D, C>& bk, Run& run, State<D, C>& st,
                                          const uint32_t (&qf)[Sh<D, C>::NW][4], const uint4* qs, const uint4* qs1, const float (&qinv)[2],
                                          unsigned char* stages, float4* rrow) {
  using X = Sh<D, C>;
  const int lane = threadIdx.x & 31, quad = lane & 3, row = lane >> 2;
  const int nt = ceil_div(run.n, kTT);
  const uint32_t vs0 = smem_addr(bk.Vs);
  // (never zero: a masked score is -infinity times it)
  const float inv[2] = {fmaxf(qinv[0] * bk.kinv, 1.17549435e-38f), fmaxf(qinv[1] * bk.kinv, 1.17549435e-38f)};
  // (queries and e^{i 8 theta} come from shared memory at every use: held in registers, they left the tile's loads and
  // products too few to overlap -- 161 us against 178 for 32 requests behind 32K tokens)
  constexpr bool BACK = X::BACK && !STK;
  const float4* e8 = bk.E8 + quad + (BACK ? X::NW * 4 : 0);
  float2 wc[X::NW], ws[X::NW];
  for (int t = 0; t < nt; ++t) {
    cp_wait<X::NST - 2>();
    __syncwarp();
    if (t % 8 == 0) {
#pragma unroll
      for (int w = 0; w < X::NW; ++w) {
        const float4 x = rrow[((quad + 4 * (w / (C / 2))) * C + 2 * (w % (C / 2))) / 2], y = bk.Ff[w * 32 + lane];
        wc[w] = make_float2((x.x * y.x - x.y * y.z) * bk.ks, (x.z * y.y - x.w * y.w) * bk.ks);
        ws[w] = make_float2((x.x * y.z + x.y * y.x) * bk.ks, (x.z * y.w + x.w * y.y) * bk.ks);
      }
    }
    const unsigned char* codes = stages + (t % X::NST) * X::STAGE;
    float sh[2][4] = {}, sl[2][4] = {};                              // products of the high parts, and the others
#pragma unroll
    for (int i = 0; i < X::NI; ++i) {
      const int P = quad + 4 * i;
      const unsigned char *e0[2], *e1[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t k0 = codes[u * X::PAGE + P * kPage + row], k1 = codes[u * X::PAGE + (P + X::NP) * kPage + row];
        e0[u] = bk.Ks + k0 * (2 * D) + P * (2 * C);
        e1[u] = bk.Ks + k1 * (2 * D) + (P + X::NP) * (2 * C);
      }
#pragma unroll
      for (int q = 0; q < (C + 7) / 8; ++q) {
        uint32_t lo[2][4], hi[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if constexpr (C == 4) {
            const uint2 x = *reinterpret_cast<const uint2*>(e0[u]), y = *reinterpret_cast<const uint2*>(e1[u]);
            lo[u][0] = x.x; lo[u][1] = x.y; hi[u][0] = y.x; hi[u][1] = y.y;
          } else {
            const uint4 x = *reinterpret_cast<const uint4*>(e0[u] + 16 * q), y = *reinterpret_cast<const uint4*>(e1[u] + 16 * q);
            lo[u][0] = x.x; lo[u][1] = x.y; lo[u][2] = x.z; lo[u][3] = x.w;
            hi[u][0] = y.x; hi[u][1] = y.y; hi[u][2] = y.z; hi[u][3] = y.w;
          }
        }
#pragma unroll
        for (int v = 0; v < (C < 8 ? C / 2 : 4); ++v) {
          const int w = i * (C / 2) + q * 4 + v;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t qh[4];
            if constexpr (STK) {
#pragma unroll
              for (int k = 0; k < 4; ++k) qh[k] = qf[w][k];
            } else {
              const uint4 x = BACK && u ? qs1[w * (X::WARP / 16)] : qs[w * 32];
              qh[0] = x.x; qh[1] = x.y; qh[2] = x.z; qh[3] = x.w;
            }
            const float2 kx = b2_lohi(lo[u][v]), ky = b2_lohi(hi[u][v]), c = wc[w], s = ws[w];
            // (scalar where a sign changes: packed operands have none to spare)
            const float2 r = make_float2(kx.x * c.x - ky.x * s.x, kx.y * c.y - ky.y * s.y);
            const float2 z = __ffma2_rn(ky, c, __fmul2_rn(kx, s));
            uint32_t rh, rl, zh, zl;
            split_h2(r, rh, rl);
            split_h2(z, zh, zl);
            mma_f16(sl[u], qh, rl, zl);
            if constexpr (!STK) {
              const uint4 x = BACK && u ? qs1[w * (X::WARP / 16) + 32] : qs[(X::NW + w) * 32];
              const uint32_t ql[4] = {x.x, x.y, x.z, x.w};
              mma_f16(sl[u], ql, rh, zh);
            }
            mma_f16(sh[u], qh, rh, zh);
            if (!BACK || u) {
              const float4 e = e8[w * 4];
              wc[w] = make_float2(c.x * e.x - s.x * e.z, c.y * e.y - s.y * e.w);
              ws[w] = __ffma2_rn(s, make_float2(e.x, e.y), __fmul2_rn(c, make_float2(e.z, e.w)));
            }
          }
        }
      }
    }
    // ---- scores -> weights: column 2 quad + k of page u; masked past the run's last token
    constexpr int NR = STK ? 1 : 2;
    const int n = min(kTT, run.n - t * kTT);
    float2 s[NR][2];                                                 // [row][page], times 1 / inv
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        s[r][u] = __fadd2_rn(make_float2(sh[u][2 * r], sh[u][2 * r + 1]), make_float2(sl[u][2 * r], sl[u][2 * r + 1]));
        if constexpr (STK) s[r][u] = __fadd2_rn(s[r][u], __fadd2_rn(make_float2(sh[u][2], sh[u][3]), make_float2(sl[u][2], sl[u][3])));
      }
    if (n < kTT) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          if (8 * u + 2 * quad >= n) s[r][u].x = -INFINITY;
          if (8 * u + 2 * quad + 1 >= n) s[r][u].y = -INFINITY;
        }
    }
    float top[NR];
    bool grow = false;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      top[r] = fmaxf(fmaxf(s[r][0].x, s[r][0].y), fmaxf(s[r][1].x, s[r][1].y));
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
      top[r] *= inv[r];
      grow = grow || top[r] > st.m[r] + 14.f;
    }
    // outputs are rescaled only when a row outgrows its reference by 2^14, so that weights stay within fp16
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float mn = top[r] > st.m[r] + 14.f ? top[r] - 6.f : st.m[r];
        const float al = ex2(st.m[r] - mn);
        st.m[r] = mn;
        st.l[r] *= al;
#pragma unroll
        for (int i = 0; i < X::NT; ++i)
#pragma unroll
          for (int k = 0; k < (STK ? 4 : 2); ++k) st.o[i][2 * r + k] *= al;
      }
    }
    uint32_t ph[4], pl[4];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float2 d = __ffma2_rn(s[r][u], make_float2(inv[r], inv[r]), make_float2(-st.m[r], -st.m[r]));   // (inv is a power of two)
        const float2 p = make_float2(ex2(d.x), ex2(d.y));
        st.l[r] += p.x + p.y;
        if constexpr (STK) split_h2(p, ph[2 * u], ph[2 * u + 1]);
        else split_h2(p, ph[2 * u + r], pl[2 * u + r]);
      }
    // ---- values.  Masked tokens take the tile's first token instead: nothing else is read
    const unsigned char* vcodes = codes + 2 * X::PAGE;
    if constexpr (C >= 8) {
      // ldmatrix hands out 8 tokens x 8 channels transposed: lane l names token l % 16, unit 2 i + l / 16
      const int tok = (lane & 15) < n ? lane & 15 : 0;
      const unsigned char* vc = vcodes + (tok >> 3) * X::PAGE + (tok & 7);
#pragma unroll
      for (int i = 0; i < X::NT / 2; ++i) {
        const int unit = 2 * i + (lane >> 4);
        const uint32_t code = vc[unit * 8 / C * kPage];
        uint32_t v[4];
        ldmatrix4_trans(v, vs0 + code * X::VROW + unit * 16);
        add_values<STK>(st.o[2 * i], ph, pl, v[0], v[1]);
        add_values<STK>(st.o[2 * i + 1], ph, pl, v[2], v[3]);
      }
    } else {
      // entries of 4 channels: lane (n, quad) takes channels [n d/8, (n + 1) d/8) of tokens 2 quad, 2 quad + 1 of
      // both pages and pairs the tokens up
      const int t0 = 2 * quad < n ? 2 * quad : 0, t1 = 2 * quad + 1 < n ? 2 * quad + 1 : 0;
      const int t2 = 8 + 2 * quad < n ? 8 + 2 * quad : 0, t3 = 9 + 2 * quad < n ? 9 + 2 * quad : 0;
      const int toks[4] = {t0, t1, t2, t3};
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {                             // 4 channels: one entry of each token
        const int grp = row * (D / 32) + q;
        uint2 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t code = vcodes[(toks[k] >> 3) * X::PAGE + grp * kPage + (toks[k] & 7)];
          v[k] = *reinterpret_cast<const uint2*>(bk.Vs + code * X::VROW + grp * 8);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t sel = i & 1 ? 0x7632u : 0x5410u;
          const uint32_t b0 = i < 2 ? __byte_perm(v[0].x, v[1].x, sel) : __byte_perm(v[0].y, v[1].y, sel);
          const uint32_t b1 = i < 2 ? __byte_perm(v[2].x, v[3].x, sel) : __byte_perm(v[2].y, v[3].y, sel);
          add_values<STK>(st.o[4 * q + i], ph, pl, b0, b1);
        }
      }
    }
    __syncwarp();                                                    // the stage is read
    if (t + X::NST - 1 < nt) fetch_tile<D, C>(g, a, run, t + X::NST - 1, stages, rrow);
    cp_commit();
  }
  cp_wait<0>();
  __syncwarp();
}

// The bf16 tokens [i0, i1) of request b's list (sink tokens, then recent ones) against NR query heads, on
// CUDA cores: D / 4 lanes to a token, a lane two frequencies (channels 2 f, 2 f + 1 and their partners) of
// the key and four channels of the value; within a batch of 8 tokens (16 at d = 64) the rotation moves on by a
// token at a time.  A batch and its RoPE row are loaded while the one before is worked on; the first one's loads
// go out together with the query's, so that an entry waits for memory once.  Row r's outputs are joined with what
// its area row holds (`fresh`: nothing yet).
template <int D, int C, int NR>
__device__ __forceinline__ void bf16_run(const Geo& g, const SharedArgs& a, const Counters& c, int b, int h, const __nv_bfloat16* q,
                                         float scale, int i0, int i1, float* area, float2* ml, bool fresh) {
  using X = Sh<D, C>;
  constexpr int LPT = D / 4, TPW = 32 / LPT, NB = 8, BT = NB * TPW;
  const int lane = threadIdx.x & 31, fp = lane % LPT, half = lane / LPT;
  const float4* rope4 = reinterpret_cast<const float4*>(a.rope);
  struct Turn { float4 x, y; };                                      // rows of the coarse and fine tables, two frequencies
  auto turn_at = [&](int p) {
    Turn t;
    t.x = __ldg(rope4 + (size_t)(p >> 3) * (X::F / 2) + fp);
    t.y = __ldg(rope4 + (size_t)(g.RC + (p & 7)) * (X::F / 2) + fp);
    return t;
  };
  auto angle = [](const Turn& t) {                                   // (cos, cos, sin, sin)
    return make_float4(t.x.x * t.y.x - t.x.y * t.y.y, t.x.z * t.y.z - t.x.w * t.y.w, t.x.x * t.y.y + t.x.y * t.y.x,
                       t.x.z * t.y.w + t.x.w * t.y.z);
  };
  const int ctx = c.ctx[b], coded = c.coded[b], S_eff = min(g.S, ctx);
  const int s1 = min(i1, S_eff), r0 = max(i0, S_eff);                // sink tokens [i0, s1), recent ones [r0, i1)
  const int nsb = max(0, ceil_div(s1 - i0, BT)), n_batch = nsb + max(0, ceil_div(i1 - r0, BT));
  const __nv_bfloat16* sk = a.sink + sink_off(g, a.layer, 0, a.step, b, h, 0);
  const __nv_bfloat16* sv = a.sink + sink_off(g, a.layer, 1, a.step, b, h, 0);
  const __nv_bfloat16* rk = a.ring + ring_off(g, a.layer, 0, a.step, b, h, 0);
  const __nv_bfloat16* rv = a.ring + ring_off(g, a.layer, 1, a.step, b, h, 0);
  // batch n: its first token of the list, how many it holds, its keys, values and rotation
  struct Batch {
    uint32_t kx[NB], ky[NB];
    uint2 v[NB];
    Turn t;
  };
  auto load = [&](int n, Batch& x) {
    const bool sink = n < nsb;
    const int t0 = sink ? i0 + n * BT : r0 + (n - nsb) * BT, end = sink ? s1 : i1;
    const __nv_bfloat16 *kb = sink ? sk : rk, *vb = sink ? sv : rv;
    int slot = sink ? t0 + half : (coded + t0 - S_eff + half) % g.R;
    // (a lane of a token past the last one may start past it: its position only has to lie within the tables)
    x.t = turn_at(min((sink ? t0 : g.S + coded + t0 - S_eff) + half, g.max_ctx - 1));
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      x.kx[u] = x.ky[u] = 0u;
      x.v[u] = make_uint2(0u, 0u);
      if (t0 + u * TPW + half < end) {
        const uint32_t* kr = reinterpret_cast<const uint32_t*>(kb + (size_t)slot * D);
        x.kx[u] = __ldg(kr + fp);
        x.ky[u] = __ldg(kr + fp + X::F / 2);
        x.v[u] = __ldg(reinterpret_cast<const uint2*>(vb + (size_t)slot * D) + fp);
      }
      slot += TPW;
      if (!sink && slot >= g.R) slot -= g.R;                          // (TPW <= R)
    }
  };
  Batch cur;
  load(0, cur);
  const Turn tq = turn_at(ctx - 1), td = turn_at(TPW);
  uint32_t qx[NR], qy[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const uint32_t* qr = reinterpret_cast<const uint32_t*>(q + (size_t)r * D);
    qx[r] = __ldg(qr + fp);
    qy[r] = __ldg(qr + fp + X::F / 2);
  }
  const float4 wq = angle(tq), dw = angle(td);
  float4 z[NR];                                                      // rotated queries: channels f, f + 1, f + d/2, f + 1 + d/2
  float m[NR], l[NR], o[NR][4];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const float2 x = b2_lohi(qx[r]), y = b2_lohi(qy[r]);
    z[r] = make_float4((x.x * wq.x - y.x * wq.z) * scale, (x.y * wq.y - y.y * wq.w) * scale, (y.x * wq.x + x.x * wq.z) * scale,
                       (y.y * wq.y + x.y * wq.w) * scale);
    m[r] = kNoMax;
    l[r] = o[r][0] = o[r][1] = o[r][2] = o[r][3] = 0.f;
  }
#pragma unroll 1
  for (int n = 0; n < n_batch; ++n) {
    Batch nxt;
    if (NR == 1 && n + 1 < n_batch) load(n + 1, nxt);              // (more rows have no registers to spare)
    const int left = (n < nsb ? s1 - i0 - n * BT : i1 - r0 - (n - nsb) * BT) - half;   // tokens from the lane's first on
    float4 w = angle(cur.t);
    float d[NR][NB];
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      const float2 x = b2_lohi(cur.kx[u]), y = b2_lohi(cur.ky[u]);
      const float k0 = x.x * w.x - y.x * w.z, k1 = x.y * w.y - y.y * w.w, k2 = y.x * w.x + x.x * w.z, k3 = y.y * w.y + x.y * w.w;
#pragma unroll
      for (int r = 0; r < NR; ++r) d[r][u] = z[r].x * k0 + z[r].y * k1 + (z[r].z * k2 + z[r].w * k3);
      w = make_float4(w.x * dw.x - w.z * dw.z, w.y * dw.y - w.w * dw.w, w.z * dw.x + w.x * dw.z, w.w * dw.y + w.y * dw.w);
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      // lane sums, transposed: a lane keeps token fp % 8 of its token group
#pragma unroll
      for (int hb = NB / 2; hb > 0; hb >>= 1) {
        const bool up = (fp & hb) != 0;
#pragma unroll
        for (int k = 0; k < hb; ++k) {
          const float send = up ? d[r][k] : d[r][k + hb], keep = up ? d[r][k + hb] : d[r][k];
          d[r][k] = keep + __shfl_xor_sync(0xffffffffu, send, hb);
        }
      }
      float s = d[r][0];
#pragma unroll
      for (int o2 = NB; o2 < LPT; o2 <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o2);
      if ((fp & (NB - 1)) * TPW >= left) s = -INFINITY;
      float top = s;
#pragma unroll
      for (int o2 = 1; o2 < NB; o2 <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o2));
      if (TPW == 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
      const float mn = fmaxf(m[r], top), al = ex2(m[r] - mn), p = ex2(s - mn);
      m[r] = mn;
      l[r] = l[r] * al + (fp < NB ? p : 0.f);
#pragma unroll
      for (int k = 0; k < 4; ++k) o[r][k] *= al;
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        const float pu = __shfl_sync(0xffffffffu, p, u + half * LPT);
        const float2 v0 = b2_lohi(cur.v[u].x), v1 = b2_lohi(cur.v[u].y);
        o[r][0] = fmaf(pu, v0.x, o[r][0]);
        o[r][1] = fmaf(pu, v0.y, o[r][1]);
        o[r][2] = fmaf(pu, v1.x, o[r][2]);
        o[r][3] = fmaf(pu, v1.y, o[r][3]);
      }
    }
    if (NR == 1) cur = nxt;
    else if (n + 1 < n_batch) load(n + 1, cur);
  }
#pragma unroll
  for (int r = 0; r < NR; ++r) {
#pragma unroll
    for (int o2 = 16; o2 > 0; o2 >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o2);
    if (TPW == 2)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[r][k] += __shfl_xor_sync(0xffffffffu, o[r][k], 16);
    float4* to = reinterpret_cast<float4*>(area + r * X::OROW) + fp;
    if (fresh) {
      if (half == 0) *to = make_float4(o[r][0], o[r][1], o[r][2], o[r][3]);
      if (lane == 0) ml[r] = make_float2(m[r], l[r]);
    } else {
      const float2 x = ml[r];
      const float M = fmaxf(m[r], x.x), f0 = ex2(x.x - M), f1 = ex2(m[r] - M);
      __syncwarp();
      if (half == 0) {
        const float4 y = *to;
        *to = make_float4(y.x * f0 + o[r][0] * f1, y.y * f0 + o[r][1] * f1, y.z * f0 + o[r][2] * f1, y.w * f0 + o[r][3] * f1);
      }
      if (lane == 0) ml[r] = make_float2(M, x.y * f0 + l[r] * f1);
    }
  }
  __syncwarp();
}

// The lane's part of row `r`'s rotated query in fragment order: D / 4 lanes to a row, lane f2 a frequency
// pair (x: its channels, y: their partners), scaled by a power of two to fp16's range.  *inv: its reciprocal.
template <int D>
__device__ __forceinline__ void query_pair(const Geo& g, const SharedArgs& a, const __nv_bfloat16* q, int p, int f2, float scale, bool live,
                                           float2& x, float2& y, float* inv) {
  constexpr int F = D / 2, LPR = D / 4;
  const float4* rope4 = reinterpret_cast<const float4*>(a.rope);
  x = y = make_float2(0.f, 0.f);
  if (live) {
    const uint32_t* qw = reinterpret_cast<const uint32_t*>(q);
    const float2 q0 = b2_lohi(__ldg(qw + f2)), q1 = b2_lohi(__ldg(qw + f2 + F / 2));
    const float4 u = __ldg(rope4 + (size_t)(p >> 3) * (F / 2) + f2), v = __ldg(rope4 + (size_t)(g.RC + (p & 7)) * (F / 2) + f2);
    const float c0 = u.x * v.x - u.y * v.y, s0 = u.x * v.y + u.y * v.x;
    const float c1 = u.z * v.z - u.w * v.w, s1 = u.z * v.w + u.w * v.z;
    x = make_float2((q0.x * c0 - q1.x * s0) * scale, (q0.y * c1 - q1.y * s1) * scale);
    y = make_float2((q1.x * c0 + q0.x * s0) * scale, (q1.y * c1 + q0.y * s1) * scale);
  }
  float mx = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y)));
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const int e = fit_exp_f(mx);
  const float qs = pow2i(e);
  x = make_float2(x.x * qs, x.y * qs);
  y = make_float2(y.x * qs, y.y * qs);
  *inv = pow2i(-e);
}

}  // namespace

// One CTA per part and KV head, 8 warps.  The step slices of the head are staged once in shared memory, the
// values as fp16 (scaled by a power of two, so that every bf16 value within 2^-28 of the largest is exact) in
// rows padded by 16 bytes (8 tokens' entries of one group then fall on different banks as often as not).
//
// What bounds it.  The bytes are few (32 requests behind 32K tokens at c = 8: 60.6 MB, 9.2 us); restoring, rotating and
// splitting a key is some 28 warp instructions a token and 16 rows, products 5 (10.6 cycles of the SM's mma.sync
// pipe), the rest weights, values and loads: 55 in all.  At 255 registers two warps share a scheduler, which issues
// 0.36 a cycle (counters: fixed latencies 0.98, shared memory 0.74, pipe throttle 0.63, instruction fetch 0.51 cycles
// of stall an instruction): 27 cycles a token and 16 rows, 157 us for those 32 requests replayed, 163 us with inputs
// that L2 does not hold.  No part of the loop bounds it by itself: without the products of the keys' or the queries'
// low parts it takes 6 or 4 % less, without bank conflicts on values 5 %; keys laid out for half their conflicts
// gained 1 %, less than laying them out cost.
// Tried and slower: 12 warps of 168 registers (spills: 214 us), values of one tile beside the scores of the next (167
// to 178), two row tiles to one restored key (156 to 173, and 99 against 86 for 64K with four heads a KV head), and
// tcgen05 products of 32 rows fed by restoring warps through swizzled shared memory (219 us: M = 128 tiles of 64
// tokens in two parts; the restoring, softmax and output warps' own instructions, 84 a token, and their hand-offs took
// 4900 cycles a tile, the tensor core 8 % of them).
template <int D, int C>
__global__ void __launch_bounds__(kShThreads, 1) shared_kernel(Geo g, SharedArgs a) {
  using X = Sh<D, C>;
  extern __shared__ __align__(128) unsigned char sm[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, quad = lane & 3, row = lane >> 2;
  const int j = blockIdx.x, h = blockIdx.y, rep = g.Hq / g.H;
  const int blk = a.step / g.Tc, step_s = a.step % g.Tc;
  unsigned char* Ks = sm;
  unsigned char* Vs = sm + X::OFF_V;
  unsigned char* area = sm + X::OFF_W + warp * X::WARP;
  float* area_f = reinterpret_cast<float*>(area);
  float4* Ff = reinterpret_cast<float4*>(sm + X::OFF_F);
  float4* E8 = reinterpret_cast<float4*>(sm + X::OFF_E);
  float4* rrow = reinterpret_cast<float4*>(sm + X::OFF_R) + warp * (X::F / 2);
  float2* ml_s = reinterpret_cast<float2*>(sm + X::OFF_ML);   // [warp][16]: rows of the area (own entries: 8, then 8 parked)
  float2* ml = ml_s + warp * kQT;
  float* inv_s = reinterpret_cast<float*>(sm + X::OFF_INV);
  uint32_t* red = reinterpret_cast<uint32_t*>(sm + X::OFF_RED);
  const uint32_t bar = smem_addr(sm + X::OFF_BAR);
  Counters c;
  c.gcum = reinterpret_cast<long long*>(sm + X::OFF_C);
  c.ocum = c.gcum + a.ng + 1;
  c.ctx = reinterpret_cast<int*>(c.ocum + a.batch + 1);
  c.coded = c.ctx + a.batch; c.own0 = c.coded + a.batch; c.gb = c.own0 + a.batch; c.sh = c.gb + a.ng + 1; c.lead = c.sh + a.ng;
  const __nv_bfloat16* kslice = a.cbp + cbp_slice_off(g, a.layer, 0, blk, h, step_s);
  const __nv_bfloat16* vslice = a.cbp + cbp_slice_off(g, a.layer, 1, blk, h, step_s);

  // before the preceding kernel has ended only L2 is touched (and nothing is read through the read-only path that
  // could move above the wait: counters and tables come by ld.global.cg)
  if (tid == 0) {
    prefetch_l2(kslice, X::KS);
    prefetch_l2(vslice, X::KS);
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  dependency_wait();
  dependents_may_launch();
  Book<D, C> bk;
  bk.Ks = Ks; bk.Vs = Vs; bk.Ff = Ff; bk.E8 = E8;
  const float4* rope4 = reinterpret_cast<const float4*>(a.rope);   // two frequencies: (cos, sin, cos, sin)
  auto pair_of = [&](int w) { return ((quad + 4 * (w / (C / 2))) * C + 2 * (w % (C / 2))) / 2; };   // lane's frequency pair w
  // the small loads first: the slices' 2 x 32 or 2 x 64 KB a CTA keep the way from L2 busy for some 2000 cycles
  const bool ok = load_counters(g, a, c, reinterpret_cast<long long*>(sm + X::OFF_P), j == 0 && h == 0);   // (its barriers publish the mbarrier)
  if (tid == 0) {
    mbar_expect_tx(bar, 2 * X::KS);
    bulk_g2s(smem_addr(Ks), kslice, X::KS, bar);
    if (!(g.fault & kFaultSharedDropSlice)) bulk_g2s(smem_addr(Vs), vslice, X::KS, bar);
  }
  // every slot of this part starts empty
  for (int i = tid; i < a.batch * rep * 2; i += kShThreads) {
    const int b = i / (rep * 2), r = i / 2 % rep;
    a.pml[(((size_t)b * g.Hq + h * rep + r) * g.max_splits + j) * 2 + (i & 1)] = make_float2(kNoMax, 0.f);
  }
  if (warp < X::NW) {
    const float4 e = __ldcg(rope4 + X::F / 2 + pair_of(warp));
    const int p = (g.S & 7) + row;
    const float4 x = __ldcg(rope4 + (size_t)(p >> 3) * (X::F / 2) + pair_of(warp));
    const float4 y = __ldcg(rope4 + (size_t)(g.RC + (p & 7)) * (X::F / 2) + pair_of(warp));
    if (row == 0) {
      E8[warp * 4 + quad] = make_float4(e.x, e.z, e.y, e.w);
      E8[(X::NW + warp) * 4 + quad] = make_float4(e.x * e.x - e.y * e.y, e.z * e.z - e.w * e.w, 2.f * e.x * e.y, 2.f * e.z * e.w);
    }
    Ff[warp * 32 + lane] = make_float4(x.x * y.x - x.y * y.y, x.z * y.z - x.w * y.w, x.x * y.y + x.y * y.x, x.z * y.w + x.w * y.z);
  }
  const float qk_scale = 1.4426950408889634f / sqrtf((float)D);
  // Fragments of a query tile: D / 4 lanes rotate a row at its own position, scale it to fp16's range and split it.
  auto set_queries = [&](const RowTile& rt) {
    uint4* Qf = reinterpret_cast<uint4*>(sm + X::OFF_Q);       // [hi, lo][k step][lane]
    constexpr int LPR = D / 4, RPW = 32 / LPR;                 // lanes of a row, rows a warp takes at once
    const int f2 = lane % LPR, P = 2 * f2 / C, sub = 2 * f2 % C / 2;
    const float4 e = __ldcg(rope4 + X::F / 2 + f2);            // e^{i 8 theta}
#pragma unroll 2
    for (int r = warp * RPW + lane / LPR; r < kQT; r += kWarps * RPW) {
      const bool live = r < rt.nrows && c.ctx[rt.request(r)] > 0;
      float2 x, y;
      float inv;
      query_pair<D>(g, a, live ? a.q + ((size_t)rt.request(r) * g.Hq + rt.head(r)) * D : a.q, live ? c.ctx[rt.request(r)] - 1 : 0, f2,
                    qk_scale, live, x, y, &inv);
      const int ks = P / 4 * (C / 2) + sub, fl = (r & 7) * 4 + P % 4, rg = r >> 3;
      auto put = [&](uint4* hi, uint4* lo) {
        uint32_t xh, xl, yh, yl;
        split_h2(x, xh, xl);
        split_h2(y, yh, yl);
        uint32_t *fh = reinterpret_cast<uint32_t*>(hi + fl), *fw = reinterpret_cast<uint32_t*>(lo + fl);
        fh[rg] = xh; fh[rg + 2] = yh;
        fw[rg] = xl; fw[rg + 2] = yl;
      };
      put(Qf + ks * 32, Qf + (X::NW + ks) * 32);
      if constexpr (X::BACK) {                                 // and turned 8 positions back, in the warps' areas
        const float2 b = make_float2(x.x * e.x + y.x * e.y, x.y * e.z + y.y * e.w);
        y = make_float2(y.x * e.x - x.x * e.y, y.y * e.z - x.y * e.w);
        x = b;
        uint4* Q1 = reinterpret_cast<uint4*>(sm + X::OFF_W + ks * X::WARP + X::PARK);
        put(Q1, Q1 + 32);
      }
      if (f2 == 0) inv_s[r] = inv;
    }
  };
  // this part of the head's list: [cut0, cut1), shared entries first; e, qt: where it begins
  const long long shared_total = ok ? c.gcum[a.ng] : 0, own_total = ok ? c.ocum[a.batch] : 0;
  const long long own_at = shared_total * kSharedWeight + (shared_total > 0 && own_total > 0 ? kOwnStage * kSharedWeight : 0);
  const long long total = own_at + own_total * kOwnWeight, at0 = div_cost(total * j, a.k), at1 = div_cost(total * (j + 1), a.k);
  const long long cut0 = min(shared_total, at0 / kSharedWeight), cut1 = min(shared_total, at1 / kSharedWeight);
  int e = a.ng, qt = 0;
  Entry en = {0, 0, 0, 0, 1};
  RowTile rt;
  rt.rep = rep; rt.h = h;
  auto next_tile = [&](bool first) {                           // moves on to the part's next query tile of shared tokens
    if (first) e = locate(c.gcum, a.ng, cut0);
    for (;; ++e, first = true) {
      if (e >= a.ng || c.gcum[e] >= cut1) { e = a.ng; return; }
      en = shared_entry(g, c, e);
      if (en.tiles == 0) continue;
      for (qt = first ? (cut0 > c.gcum[e] ? (int)div_cost(cut0 - c.gcum[e], en.each()) : 0) : qt + 1; qt < en.qtiles; ++qt) {
        const long long base = c.gcum[e] + qt * en.each() + en.fixed;
        if (base >= cut1) { e = a.ng; return; }
        if (max(0ll, cut0 - base) < min((long long)en.tiles, cut1 - base)) {
          rt.b0 = c.gb[e];
          rt.r0 = qt * kQT;
          rt.nrows = min(kQT, (c.gb[e + 1] - c.gb[e]) * rep - rt.r0);
          return;
        }
      }
    }
  };
  // the warp's share of the query tile's tokens, its first codes on their way
  Run run;
  auto start_shared = [&]() {
    const long long base = c.gcum[e] + qt * en.each() + en.fixed;
    const int t0 = (int)max(0ll, cut0 - base), t1 = (int)min((long long)en.tiles, cut1 - base);
    const int w0 = t0 + (int)((long long)(t1 - t0) * warp / kWarps), w1 = t0 + (int)((long long)(t1 - t0) * (warp + 1) / kWarps);
    run.lead = c.lead[e];
    run.pg0 = 2 * w0;
    run.n = w0 < w1 ? min(w1 * kTT, c.sh[e]) - w0 * kTT : 0;
    run.pg_end = run.pg0 + ceil_div(run.n, kPage);
    run.kcode = a.idx + idx_page_off(g, a.layer, blk, run.lead, h, 0, 0);
    run.vcode = a.idx + idx_page_off(g, a.layer, blk, run.lead, h, 1, 0);
    run.ids = 0; run.ids_at = -32;
    begin_run<D, C>(g, a, run, area, rrow);
  };
  if (ok) {
    next_tile(true);
    if (e < a.ng) {
      start_shared();
      set_queries(rt);
    }
    if (g.pool) check_rows(g, a, c);
  }
  const bool late = __syncthreads_or(!mbar_wait(bar, 0, g.wait_iters));
  if (late || !ok) {
    if (late && tid == 0) {
      set_status(a.st, LVQ_ETIMEOUT);
      if (g.fault & kFaultSharedDropSlice) bulk_g2s(smem_addr(Vs), vslice, X::KS, bar);   // (the barrier expects it)
      mbar_wait(bar, 0, kWaitIters);                           // the copies land before the CTA exits
    }
    cp_wait<0>();
    return;
  }
  // the slices' largest finite magnitudes (as bf16 pairs); the values go to their padded rows as scaled fp16
  {
    constexpr int NV = X::KS / 16 / kShThreads, VPR = D / 8;   // vectors of a thread, of a row
    // (a NaN never wins a maximum; an infinity, below, counts nothing)
    auto amax = [](uint4 w, __nv_bfloat162 m) {
      auto mag = [](uint32_t x) { return __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x)); };
      return __hmax2(m, __hmax2(__hmax2(mag(w.x), mag(w.y)), __hmax2(mag(w.z), mag(w.w))));
    };
    auto widest = [](__nv_bfloat162 m) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(&m);
      return max(w & 0xffffu, w >> 16);
    };
    auto finite = [](uint32_t w) {
      w &= 0x7fff7fffu;
      return max((w & 0xffffu) < 0x7f80u ? w & 0xffffu : 0u, (w >> 16) < 0x7f80u ? w >> 16 : 0u);
    };
    __nv_bfloat162 k2 = __floats2bfloat162_rn(0.f, 0.f), v2 = k2;
    uint4 v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = reinterpret_cast<const uint4*>(Vs)[tid + i * kShThreads];
      v2 = amax(v[i], v2);
    }
#pragma unroll 4
    for (int i = 0; i < NV; ++i) k2 = amax(reinterpret_cast<const uint4*>(Ks)[tid + i * kShThreads], k2);
    uint32_t ka = widest(k2), va = widest(v2);
    if (__any_sync(0xffffffffu, max(ka, va) >= 0x7f80u)) {
      ka = va = 0;
#pragma unroll 1
      for (int i = tid; i < X::KS / 16; i += kShThreads) {
        const uint4 k = reinterpret_cast<const uint4*>(Ks)[i], x = reinterpret_cast<const uint4*>(Vs)[i];
        ka = max(ka, max(max(finite(k.x), finite(k.y)), max(finite(k.z), finite(k.w))));
        va = max(va, max(max(finite(x.x), finite(x.y)), max(finite(x.z), finite(x.w))));
      }
    }
    ka = __reduce_max_sync(0xffffffffu, ka);
    va = __reduce_max_sync(0xffffffffu, va);
    if (lane == 0) { red[warp] = ka; red[kWarps + warp] = va; }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) { ka = max(ka, red[w]); va = max(va, red[kWarps + w]); }
    bk.ks = pow2i(fit_exp(ka));
    bk.kinv = pow2i(-fit_exp(ka));
    const float vscale = pow2i(fit_exp(va) + 1);
    // (every vector is in registers: the rows are spread out in place)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = tid + i * kShThreads;
      auto cv = [&](uint32_t x) { return pack_h2(bf16_lo(x) * vscale, bf16_hi(x) * vscale); };
      *(reinterpret_cast<uint4*>(Vs + (at / VPR) * X::VROW) + at % VPR) = make_uint4(cv(v[i].x), cv(v[i].y), cv(v[i].z), cv(v[i].w));
    }
    if (tid == 0) red[2 * kWarps] = __float_as_uint(pow2i(-fit_exp(va) - 1));
    __syncthreads();
  }
  const float vback = __uint_as_float(red[2 * kWarps]);
  auto slot_of = [&](int b, int hq, int kind) { return (((size_t)b * g.Hq + hq) * g.max_splits + j) * 2 + kind; };

  // ---- shared entries: the CTA's warps share out the tiles of one query tile at a time
  while (e < a.ng) {
    {
      const float qinv[2] = {inv_s[row], inv_s[row + 8]};
      State<D, C> st;
      st.clear();
      const uint32_t none[X::NW][4] = {};
      if (run.n > 0) coded_run<D, C, false>(g, a, bk, run, st, none, reinterpret_cast<const uint4*>(sm + X::OFF_Q) + lane,
                                               reinterpret_cast<const uint4*>(sm + X::OFF_W + X::PARK) + lane, qinv, area, rrow);
      if constexpr (X::BACK) __syncthreads();                  // (queries lie in the areas)
      // the warps' results are joined
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 1);
        st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 2);
        if (quad == 0) ml[row + 8 * r] = make_float2(st.m[r], st.l[r]);
        float* to = area_f + (row + 8 * r) * X::OROW;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < X::NT; ++i) to[out_channel<D, C>(i, 2 * quad + n)] = st.o[i][2 * r + n];
      }
      __syncthreads();
      {
        constexpr int TPR = kShThreads / kQT, CH = D / TPR;    // threads of a row, channels of a thread
        const int r = tid / TPR, c0 = tid % TPR * CH;
        if (r < rt.nrows && c.ctx[rt.request(r)] > 0) {
          float M = kNoMax, L = 0.f, o[CH] = {};
#pragma unroll
          for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml_s[w * kQT + r].x);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 x = ml_s[w * kQT + r];
            const float f = ex2(x.x - M);
            L += f * x.y;
            const float* from = reinterpret_cast<const float*>(sm + X::OFF_W + w * X::WARP) + r * X::OROW + c0;
#pragma unroll
            for (int i = 0; i < CH; ++i) o[i] += f * from[i];
          }
          const size_t slot = slot_of(rt.request(r), rt.head(r), 0);
#pragma unroll
          for (int i = 0; i < CH; i += 4)
            *reinterpret_cast<float4*>(a.po + slot * D + c0 + i) =
                make_float4(o[i] * vback, o[i + 1] * vback, o[i + 2] * vback, o[i + 3] * vback);
          if (c0 == 0) a.pml[slot] = make_float2(M, L);
        }
      }
      next_tile(false);
      __syncthreads();                                         // the areas are read
      if (e < a.ng) {
        start_shared();
        set_queries(rt);
        __syncthreads();
      }
    }
  }

  // ---- own entries: a contiguous run of the part's tiles to a warp
  const long long o0 = div_cost(max(0ll, at0 - own_at), kOwnWeight), o1 = div_cost(max(0ll, at1 - own_at), kOwnWeight);
  if (o0 >= o1) return;
  const long long x0 = o0 + (o1 - o0) * warp / kWarps, x1 = o0 + (o1 - o0) * (warp + 1) / kWarps;
  int* park_s = reinterpret_cast<int*>(red) + 2 * kWarps;      // [warp]: entry tile whose beginning another warp has, or -1
  int* last_s = reinterpret_cast<int*>(red) + kWarps;          // [warp]: its last tile of that entry ends the part's share
  int park = -1, open = -1, open_b = 0, open_qt = 0, ended = 0, any = 0;   // open: the last piece, which other warps continue
  __syncthreads();                                             // (red is reused)
  if (x0 < x1) {
    for (int b = locate(c.ocum, a.batch, x0); b < a.batch && c.ocum[b] < x1; ++b) {
      const Entry en = own_entry(g, c, b);
      if (en.tiles == 0) continue;
      const long long eat = c.ocum[b];
      for (int qt = x0 > eat ? (int)min((long long)en.qtiles, div_cost(x0 - eat, en.each())) : 0; qt < en.qtiles; ++qt) {
        const long long base = eat + qt * en.each() + en.fixed;
        if (base >= x1) break;
        auto tile = [&](long long x) { return en.tile_at((int)min((long long)en.units(), max(0ll, x - base))); };
        const int ta = tile(x0), tb = tile(x1);
        if (ta >= tb) continue;
        const int Ta = tile(o0), Tb = tile(o1);                // the part's share
        any = 1;
        const int nrows = min(kOT, rep - qt * kOT);
        const __nv_bfloat16* q = a.q + ((size_t)b * g.Hq + h * rep + qt * kOT) * D;
        const int own0 = c.own0[b], rest = c.coded[b] - own0, nc = ceil_div(rest, kTT);
        const bool coded = ta < nc;
        if (coded) {
          run.lead = b;
          run.pg0 = own0 / kPage + 2 * ta;
          run.n = min(min(tb, nc) * kTT, rest) - ta * kTT;
          run.pg_end = run.pg0 + ceil_div(run.n, kPage);
          run.kcode = a.idx + idx_page_off(g, a.layer, blk, b, h, 0, 0);
          run.vcode = a.idx + idx_page_off(g, a.layer, blk, b, h, 1, 0);
          run.ids = 0; run.ids_at = -32;
          // fragments [k step][lane], high parts in registers 0, 2, low in 1, 3: of up to two rows in a place of their own,
          // so that the codes can be on their way meanwhile; of more in the stages
          const bool small = nrows <= 2;
          uint4* Qf = small ? reinterpret_cast<uint4*>(sm + X::OFF_Q) + warp * (X::NW * 8) : reinterpret_cast<uint4*>(area);
          const int ql = small ? 8 : 32;
          if (small) begin_run<D, C>(g, a, run, area, rrow);
          constexpr int LPR = D / 4, RPW = 32 / LPR;
          const int f2 = lane % LPR, P = 2 * f2 / C, sub = 2 * f2 % C / 2;
          for (int r0 = 0; r0 < nrows; r0 += RPW) {
            const int r = r0 + lane / LPR;
            float2 x, y;
            float inv;
            query_pair<D>(g, a, q + (size_t)min(r, nrows - 1) * D, c.ctx[b] - 1, f2, qk_scale, true, x, y, &inv);
            uint4 f;
            split_h2(x, f.x, f.y);
            split_h2(y, f.z, f.w);
            if (r < nrows) {
              Qf[(P / 4 * (C / 2) + sub) * ql + r * 4 + P % 4] = f;
              if (f2 == 0) ml[r].x = inv;
            }
          }
          __syncwarp();
          uint32_t qf[X::NW][4];
#pragma unroll
          for (int w = 0; w < X::NW; ++w) {
            const uint4 u = row < nrows ? Qf[w * ql + lane] : make_uint4(0u, 0u, 0u, 0u);
            qf[w][0] = u.x; qf[w][1] = u.y; qf[w][2] = u.z; qf[w][3] = u.w;
          }
          const float qi = row < nrows ? ml[row].x : 1.f;
          const float qinv[2] = {qi, qi};
          __syncwarp();
          State<D, C> st;
          st.clear();
          if (!small) begin_run<D, C>(g, a, run, area, rrow);
          coded_run<D, C, true>(g, a, bk, run, st, qf, nullptr, nullptr, qinv, area, rrow);
          st.l[0] += __shfl_xor_sync(0xffffffffu, st.l[0], 1);
          st.l[0] += __shfl_xor_sync(0xffffffffu, st.l[0], 2);
          if (row < nrows) {
            if (quad == 0) ml[row] = make_float2(st.m[0], st.l[0]);
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int i = 0; i < X::NT; ++i)
                area_f[row * X::OROW + out_channel<D, C>(i, 2 * quad + n)] = (st.o[i][n] + st.o[i][2 + n]) * vback;
          }
          __syncwarp();
        }
        if (tb > nc) {
          const int i0 = max(ta - nc, 0) * kTT, i1 = min((tb - nc) * kTT, c.ctx[b] - c.coded[b]);
          int r = 0;
          for (; r + 4 <= nrows; r += 4)
            bf16_run<D, C, 4>(g, a, c, b, h, q + (size_t)r * D, qk_scale, i0, i1, area_f + r * X::OROW, ml + r, !coded);
          for (; r < nrows; ++r)
            bf16_run<D, C, 1>(g, a, c, b, h, q + (size_t)r * D, qk_scale, i0, i1, area_f + r * X::OROW, ml + r, !coded);
        }
        const int id = b * en.qtiles + qt;
        if (ta > Ta) {
          // another warp has the beginning: parked for it
          for (int r = 0; r < nrows; ++r)
            for (int i = lane; i < D; i += 32) area_f[X::PARK / 4 + r * X::OROW + i] = area_f[r * X::OROW + i];
          if (lane < nrows) ml[kOT + lane] = ml[lane];
          park = id;
          ended = tb == Tb;
        } else if (tb < Tb) {
          open = id;
          open_b = b; open_qt = qt;
        } else {
          for (int r = 0; r < nrows; ++r) {
            const size_t slot = slot_of(b, h * rep + qt * kOT + r, 1);
            for (int i = lane; i < D / 4; i += 32)
              *reinterpret_cast<float4*>(a.po + slot * D + 4 * i) = *reinterpret_cast<const float4*>(area_f + r * X::OROW + 4 * i);
            if (lane == 0) a.pml[slot] = ml[r];
          }
        }
        __syncwarp();
      }
    }
  }
  if (lane == 0) {
    park_s[warp] = any ? park : -2;                            // -2: no tile at all
    last_s[warp] = ended;
  }
  __syncthreads();
  if (open >= 0) {
    const int nrows = min(kOT, rep - open_qt * kOT);
    for (int r = 0; r < nrows; ++r) {
      float M = ml[r].x, L = 0.f;
      int wl = warp;                                           // warps (warp, wl] continue the entry
      for (int w = warp + 1; w < kWarps; ++w) {
        if (park_s[w] == -2) continue;
        if (park_s[w] != open) break;
        wl = w;
        M = fmaxf(M, ml_s[w * kQT + kOT + r].x);
        if (last_s[w]) break;
      }
      const size_t slot = slot_of(open_b, h * rep + open_qt * kOT + r, 1);
      float o[D / 32];
      const float f0 = ex2(ml[r].x - M);
      L = ml[r].y * f0;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = area_f[r * X::OROW + lane + 32 * i] * f0;
      for (int w = warp + 1; w <= wl; ++w) {
        if (park_s[w] != open) continue;
        const float2 x = ml_s[w * kQT + kOT + r];
        const float f = ex2(x.x - M);
        L += f * x.y;
        const float* from = reinterpret_cast<const float*>(sm + X::OFF_W + w * X::WARP + X::PARK) + r * X::OROW;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] += f * from[lane + 32 * i];
      }
#pragma unroll
      for (int i = 0; i < D / 32; ++i) a.po[slot * D + lane + 32 * i] = o[i];
      if (lane == 0) a.pml[slot] = make_float2(M, L);
    }
  }
}

// Joins the partials of a (request, query head): a warp each, a lane d / 32 channels.
template <int D>
__global__ void __launch_bounds__(128) shared_merge_kernel(Geo g, int rows, int k, const float* po, const float2* pml, float* out,
                                                           float* lse) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  const long long r = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  dependency_wait();
  dependents_may_launch();
  if (r >= rows) return;
  const size_t slot0 = (size_t)r * g.max_splits * 2;
  constexpr int NS = 4;                                        // slots of a lane kept in registers: 128 in all
  float2 x[NS];
  float M = kNoMax;
#pragma unroll
  for (int u = 0; u < NS; ++u) x[u] = 32 * u + lane < 2 * k ? __ldcg(pml + slot0 + 32 * u + lane) : make_float2(kNoMax, 0.f);
#pragma unroll
  for (int u = 0; u < NS; ++u)
    if (x[u].y != 0.f) M = fmaxf(M, x[u].x);
  for (int i = 32 * NS + lane; i < 2 * k; i += 32) {
    const float2 y = __ldcg(pml + slot0 + i);
    if (y.y != 0.f) M = fmaxf(M, y.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float den = 0.f, acc[V] = {};
  auto add = [&](float2 y, int i0) {                           // slots i0 .. i0 + 31, one a lane
    const float w = y.y != 0.f ? ex2(y.x - M) : 0.f;
    den += w * y.y;
    unsigned todo = __ballot_sync(0xffffffffu, y.y != 0.f);
    while (todo) {                                             // four partials at a time, in slot order
      float f[4];
      float v[4][V];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = todo ? __ffs(todo) - 1 : -1;
        todo &= todo - 1;
        f[u] = __shfl_sync(0xffffffffu, w, i < 0 ? 0 : i);
        if (i < 0) f[u] = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) v[u][e] = i < 0 ? 0.f : __ldcg(po + (slot0 + i0 + i) * D + lane * V + e);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = fmaf(f[u], v[u][e], acc[e]);
    }
  };
#pragma unroll
  for (int u = 0; u < NS; ++u)
    if (32 * u < 2 * k) add(x[u], 32 * u);
  for (int i0 = 32 * NS; i0 < 2 * k; i0 += 32) add(i0 + lane < 2 * k ? __ldcg(pml + slot0 + i0 + lane) : make_float2(kNoMax, 0.f), i0);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
#pragma unroll
  for (int e = 0; e < V; ++e) out[(size_t)r * D + lane * V + e] = den != 0.f ? acc[e] / den : 0.f;
  if (lane == 0) lse[r] = den != 0.f ? (M + log2f(den)) * 0.6931471805599453f : -INFINITY;
}

template <int D, int C>
static cudaError_t shared_as(const Geo& g, SharedArgs a, float* out, float* lse, cudaStream_t s) {
  static bool attr_set[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !attr_set[dev]) {
    e = cudaFuncSetAttribute(shared_kernel<D, C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Sh<D, C>::smem(kSharedMaxBatch, kSharedMaxBatch));
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) attr_set[dev] = true;
  }
  // both kernels may start while the one before them ends, and wait for it before they read or write anything
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(a.k, g.H);
  lc.blockDim = dim3(kShThreads);
  lc.dynamicSmemBytes = Sh<D, C>::smem(a.batch, a.ng);
  lc.stream = s;
  lc.attrs = attr;
  lc.numAttrs = 1;
  e = cudaLaunchKernelEx(&lc, shared_kernel<D, C>, g, a);
  if (e != cudaSuccess) return e;
  const int rows = a.batch * g.Hq;
  lc.gridDim = dim3((rows + 3) / 4);
  lc.blockDim = dim3(128);
  lc.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&lc, shared_merge_kernel<D>, g, rows, a.k, (const float*)a.po, (const float2*)a.pml, out, lse);
}

int shared_parts(const Geo& g, int batch, int n_sm) {
  // one wave of CTAs; where the layout holds few tokens, two parts a request and two for the shared ones, or one to
  // 128 tokens (two requests of 464 tokens, one head: 12.3 us with 9 parts, 15.5 with 64, 19.0 with one; four of 20
  // tokens, 16 heads: 13.9 with 9, 18.2 with one)
  const long long by_tokens = ((long long)batch * g.max_ctx + 127) / 128, by_batch = 2ll * batch + 2;
  const long long most = by_tokens > by_batch ? by_tokens : by_batch;
  int k = n_sm / g.H < 1 ? 1 : n_sm / g.H;
  if (k > g.max_splits) k = g.max_splits;
  if (k > most) k = (int)most;
  return k;
}

bool shared_rows_countable(const Geo& g, int batch, int k) {
  return !g.pool || (g.P / ((long long)k * g.H) + 1) * (batch - 1) <= 1 << 30;   // (check_rows)
}

cudaError_t launch_decode_shared(const Geo& g, int layer, int step, int batch, const __nv_bfloat16* q,
                                 const int32_t* ctx_len, const int32_t* coded_len, int n_groups,
                                 const int32_t* group_begin, const int32_t* group_tokens, const __nv_bfloat16* sink,
                                 const __nv_bfloat16* ring, const uint8_t* idx, const __nv_bfloat16* cbp,
                                 const float* rope, int k, float* ws, float* out, float* lse, int32_t* st,
                                 cudaStream_t s) {
  SharedArgs a = {layer, step, batch, n_groups, k, q, ctx_len, coded_len, group_begin, group_tokens,
                  sink, ring, idx, cbp, rope, ws, nullptr, st};
  a.pml = reinterpret_cast<float2*>(ws + (size_t)g.B * g.Hq * g.max_splits * 2 * g.d);
  if (g.d == 128 && g.c == 4) return shared_as<128, 4>(g, a, out, lse, s);
  if (g.d == 128 && g.c == 8) return shared_as<128, 8>(g, a, out, lse, s);
  if (g.d == 128 && g.c == 16) return shared_as<128, 16>(g, a, out, lse, s);
  if (g.d == 64 && g.c == 4) return shared_as<64, 4>(g, a, out, lse, s);
  if (g.d == 64 && g.c == 8) return shared_as<64, 8>(g, a, out, lse, s);
  return cudaErrorInvalidValue;
}

}  // namespace lvq
