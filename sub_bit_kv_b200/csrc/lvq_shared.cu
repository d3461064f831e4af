// Decode attention for groups of requests that share coded prefixes.
//
// "LoopVQ summary", section "premises and limits": the attention reads only the step-t slice of
// each codebook, splits the coded tokens and merges the splits, and the bf16 sink and recent
// tokens, by logsumexp; section "how it differs": RoPE is applied to the reconstructed key.  Here
// the coded tokens that a group's requests have in common are restored and rotated once, and
// scored against every query of the group.
//
// Work.  A KV head's work is a list of entries: for every group its shared tokens, once per tile of
// kQT query rows (request, query head of the KV head); then for every request its own tokens (sink,
// the rest of its coded tokens, recent window), once per tile of its query heads.  An entry costs
// its 16-token tiles and a fixed overhead per query tile; the list is cut into k parts of equal
// cost, and CTA (j, h) takes part j of KV head h.  Every CTA derives the same cut from the
// counters.  Per entry it covers, a CTA leaves one partial (m, l, o) per query row; every row has a
// slot per part and kind (shared, own), and the merge kernel joins the ones that are not empty in
// a fixed order.
#include <cuda_fp16.h>

#include "lvq_common.cuh"

namespace lvq {

namespace {

constexpr int kQT = 16;                 // query rows of a tile
constexpr int kTT = 16;                 // tokens of a tile
constexpr int kOverhead = 20;           // fixed cost of an entry's query tile, in token tiles
constexpr int kWarps = 8;
constexpr int kShThreads = 32 * kWarps;

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

// Counters of the batch in shared memory (the partition's inputs).
struct Counters {
  int *ctx, *coded, *own0;              // [batch]: context (0: unusable), coded tokens, shared tokens of its group
  int *gb, *sh, *lead;                  // [ng + 1], [ng], [ng]: first request, shared tokens, first usable request
};

__device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Entries 0 .. ng-1: the groups' shared tokens; ng .. ng+batch-1: the requests' own tokens.
struct Entry {
  int tiles, qtiles;                    // token tiles, query tiles
  __device__ long long cost() const { return tiles ? (long long)qtiles * (kOverhead + tiles) : 0; }
};
__device__ inline Entry entry_of(const Geo& g, const Counters& c, int ng, int e) {
  const int rep = g.Hq / g.H;
  if (e < ng) return {c.sh[e] / kTT + (c.sh[e] % kTT != 0), ceil_div((c.gb[e + 1] - c.gb[e]) * rep, kQT)};
  const int b = e - ng, ctx = c.ctx[b];
  const int S_eff = min(g.S, ctx), recent = ctx - S_eff - c.coded[b];
  return {ceil_div(S_eff, kTT) + ceil_div(c.coded[b] - c.own0[b], kTT) + ceil_div(recent, kTT), ceil_div(rep, kQT)};
}

// Loads and checks the counters; returns false (for every thread) if group_begin is not as described.
__device__ bool load_counters(const Geo& g, const SharedArgs& a, Counters& c, bool report) {
  const int tid = threadIdx.x;
  bool ok = true;
  for (int i = tid; i <= a.ng; i += kShThreads) {
    const int v = __ldg(a.gb + i);
    c.gb[i] = v;
    ok = ok && v >= 0 && v <= a.batch && (i > 0 || v == 0) && (i < a.ng || v == a.batch);
    if (i < a.ng) {
      ok = ok && __ldg(a.gb + i + 1) >= v;
      c.sh[i] = max(0, __ldg(a.gt + i)) / kPage * kPage;
      c.lead[i] = a.batch;
    }
  }
  for (int b = tid; b < a.batch; b += kShThreads) {
    const int ctx = __ldg(a.ctx_len + b), L = __ldg(a.coded_len + b);
    const int recent = ctx - min(g.S, max(ctx, 0)) - L;
    const bool bad = ctx < 1 || ctx > g.max_ctx || L < 0 || L > g.P * kPage || (L > 0 && ctx < g.S + L) || recent < 0 ||
                     recent > g.R;
    if (bad && report) set_status(a.st, LVQ_ECAPACITY);
    c.ctx[b] = bad ? 0 : ctx;
    c.coded[b] = bad ? 0 : L;
  }
  if (__syncthreads_or(!ok)) {
    if (tid == 0 && report) set_status(a.st, LVQ_EINVAL);
    return false;
  }
  // a group shares no more than its shortest usable request has coded
  auto group_of = [&](int b) {
    int lo = 0, hi = a.ng;                       // the last group that begins at or before b
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (c.gb[mid] <= b) lo = mid; else hi = mid;
    }
    return lo;
  };
  for (int b = tid; b < a.batch; b += kShThreads)
    if (c.ctx[b] > 0) {
      atomicMin(&c.sh[group_of(b)], c.coded[b] / kPage * kPage);
      atomicMin(&c.lead[group_of(b)], b);
    }
  __syncthreads();
  for (int b = tid; b < a.batch; b += kShThreads) c.own0[b] = c.ctx[b] > 0 ? c.sh[group_of(b)] : 0;
  for (int e = tid; e < a.ng; e += kShThreads)
    if (c.lead[e] == a.batch) c.sh[e] = 0;       // no usable request
  __syncthreads();
  return true;
}

// Pool mode: the rows of a group name the same pages for its shared tokens.  The CTAs share the comparison.
__device__ void check_rows(const Geo& g, const SharedArgs& a, const Counters& c) {
  const int n_thr = gridDim.x * gridDim.y * kShThreads, me = (blockIdx.y * gridDim.x + blockIdx.x) * kShThreads + threadIdx.x;
  bool ok = true;
  for (int e = 0; e < a.ng; ++e)
    for (int b = c.lead[e] + 1; b < c.gb[e + 1]; ++b) {
      if (c.ctx[b] == 0) continue;
      const int32_t *x = g.pt + (size_t)c.lead[e] * g.pts, *y = g.pt + (size_t)b * g.pts;
      for (int p = me; p < c.sh[e] / kPage; p += n_thr) ok = ok && __ldg(x + p) == __ldg(y + p);
    }
  if (!ok) set_status(a.st, LVQ_EINVAL);
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
  static constexpr int PAGE = NG * kPage;          // bytes of one K (or V) page
  static constexpr int STAGE = 4 * PAGE;           // a tile's codes: K pages, V pages
  static constexpr int KS = kEntries * D * 2;      // a step slice
  static constexpr int VROW = D * 2 + 16;          // a padded row of the value slice
  static constexpr int OROW = D + 4;               // a padded row of a warp's output, in floats
  static constexpr int WARP = kQT * OROW * 4;      // a warp's area: code stages or bf16 rows, then its output
  static constexpr int NST = WARP / STAGE < 6 ? WARP / STAGE : 6;
  static constexpr int OFF_V = KS;
  static constexpr int OFF_W = OFF_V + kEntries * VROW;
  static constexpr int OFF_Q = OFF_W + kWarps * WARP;
  static constexpr int OFF_F = OFF_Q + 2 * NW * 32 * 16;
  static constexpr int OFF_ML = OFF_F + NW * 32 * 16;
  static constexpr int OFF_INV = OFF_ML + kWarps * kQT * 8;
  static constexpr int OFF_RED = OFF_INV + kQT * 4;
  static constexpr int OFF_BAR = OFF_RED + 2 * kWarps * 4;
  static constexpr int OFF_CUT = OFF_BAR + 16;
  static constexpr int OFF_C = OFF_CUT + 32;
  static constexpr int smem(int batch, int ng) { return OFF_C + (3 * batch + 3 * ng + 1) * 4; }
  static_assert(NP % 4 == 0 && NI * C == 2 * NW, "lane mapping");
  static_assert(NST >= 3 && kWarps * WARP >= KS && WARP >= 2 * kTT * D * 2, "the warps' areas");
  static_assert(OFF_C + (6 * kSharedMaxBatch + 1) * 4 <= 227 * 1024, "shared memory");
  static_assert(OFF_W % 16 == 0 && OFF_BAR % 8 == 0 && OFF_CUT % 8 == 0, "alignment");
};

__device__ inline uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ inline uint32_t pack_b2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ inline float2 unpack_h2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
// a pair of values as the sum of two fp16 pairs: hi + lo, good to 2^-22 of each value (2^-25 at least)
__device__ inline void split_h2(float2 v, uint32_t& hi, uint32_t& lo) {
  hi = pack_h2(v.x, v.y);
  const float2 b = unpack_h2(hi);
  const float2 r = __fadd2_rn(v, make_float2(-b.x, -b.y));
  lo = pack_h2(r.x, r.y);
}
__device__ inline float2 neg2(float2 v) { return make_float2(-v.x, -v.y); }

__device__ inline void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ inline void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// 2^e as a float, e clamped to the normal range
__device__ inline float pow2i(int e) { return __int_as_float((min(max(e, -126), 127) + 127) << 23); }
// the largest finite magnitude of a bf16 pair, as the bits of a bf16 (infinities and NaN count nothing)
__device__ inline uint32_t amax_b2(uint32_t w, uint32_t m) {
  const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
  m = max(m, lo < 0x7f80u ? lo : 0u);
  return max(m, hi < 0x7f80u ? hi : 0u);
}
// the power of two that brings magnitudes up to that bf16 below 2^14 (none where all are zero; its reciprocal
// and its products with weights up to 2^14 stay normal floats)
__device__ inline int fit_exp(uint32_t bits) { return bits ? min(13 - ((int)(bits >> 7) - 127), 90) : 0; }

// A warp's running softmax over its tokens, for the 16 rows of the query tile: lane (r, quad) holds rows
// r and r + 8.  m is a reference no more than 2^14 below the largest weight: p = 2^(s - m).
template <int D, int C>
struct State {
  float o[Sh<D, C>::NT][4];
  float m[2], l[2];
};

// Scores of a token tile -> weights (and their sums); the outputs are rescaled only when a row's largest
// score outgrows its reference by 2^14, so that weights stay within fp16.
template <int D, int C>
__device__ inline void softmax_tile(State<D, C>& st, float (&s)[2][4], const float (&inv)[2], int n, int quad) {
  if (n < kTT) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[u][k] = 8 * u + 2 * quad + (k & 1) < n ? s[u][k] * inv[k >> 1] : -INFINITY;
  } else {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[u][k] *= inv[k >> 1];
  }
  float t[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    t[r] = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
    t[r] = fmaxf(t[r], __shfl_xor_sync(0xffffffffu, t[r], 1));
    t[r] = fmaxf(t[r], __shfl_xor_sync(0xffffffffu, t[r], 2));
  }
  if (__any_sync(0xffffffffu, t[0] > st.m[0] + 14.f || t[1] > st.m[1] + 14.f)) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float mn = t[r] > st.m[r] + 14.f ? t[r] - 6.f : st.m[r];
      const float al = ex2(st.m[r] - mn);
      st.m[r] = mn;
      st.l[r] *= al;
#pragma unroll
      for (int i = 0; i < Sh<D, C>::NT; ++i) { st.o[i][2 * r] *= al; st.o[i][2 * r + 1] *= al; }
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s[u][k] = ex2(s[u][k] - st.m[k >> 1]);
      st.l[k >> 1] += s[u][k];
    }
}

// Rotates the lane's frequency pair of one token (x: channels f, f + 1; y: their partners f + d/2, ...) by
// (c, s) and accumulates its products with the query fragments: three products of two-part operands, the
// smallest (lo x lo) left out.
__device__ inline void score_pair(float (&acc)[4], float2 x, float2 y, float2 c, float2 s, float2 ns, const uint32_t (&qh)[4],
                                  const uint32_t (&ql)[4]) {
  const float2 r = __ffma2_rn(x, c, __fmul2_rn(y, ns));
  const float2 t = __ffma2_rn(y, c, __fmul2_rn(x, s));
  uint32_t rh, rl, th, tl;
  split_h2(r, rh, rl);
  split_h2(t, th, tl);
  mma_f16(acc, qh, rl, tl);
  mma_f16(acc, ql, rh, th);
  mma_f16(acc, qh, rh, th);
}

__device__ inline float2 b2_lohi(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }

}  // namespace

// One CTA per part and KV head, 8 warps.  The step slices of the head are staged once in shared memory, the
// values as fp16 (scaled by a power of two, so that every bf16 value within 2^-28 of the largest is exact).
// The tokens of a part are shared out over the warps in contiguous runs of 16-token tiles; a warp keeps its
// own running softmax and outputs in registers, and the warps are joined at the end of an entry.
//
// Per tile, lane (j, quad) restores token j of each of the two pages: the entries of pair-groups
// P = quad + 4 i straight into the B fragments of mma.sync m16n8k16 (the order of a dot product's channels is
// free, so a fragment's k indices are the channels of the lane's own entries), rotated in fp32 by
// e^{i p theta}, which moves on by one page (8 positions) with one complex multiplication.  Keys and queries
// enter as sums of two fp16 values.  The value fragments need the channels in the lane's row instead: lane
// (n, quad) takes channels [n d/8, (n + 1) d/8) of tokens 2 quad, 2 quad + 1 of both pages.
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
  uint4* Qf = reinterpret_cast<uint4*>(sm + X::OFF_Q);        // [hi, lo][k step][lane]
  float4* Ff = reinterpret_cast<float4*>(sm + X::OFF_F);      // [frequency pair][lane]: (cos, cos, sin, sin) at S % 8 + j
  float2* ml = reinterpret_cast<float2*>(sm + X::OFF_ML);     // [warp][row]
  float* inv_s = reinterpret_cast<float*>(sm + X::OFF_INV);   // [row]
  uint32_t* red = reinterpret_cast<uint32_t*>(sm + X::OFF_RED);
  long long* cut = reinterpret_cast<long long*>(sm + X::OFF_CUT);
  const uint32_t bar = smem_addr(sm + X::OFF_BAR);
  Counters c;
  c.ctx = reinterpret_cast<int*>(sm + X::OFF_C);
  c.coded = c.ctx + a.batch; c.own0 = c.coded + a.batch; c.gb = c.own0 + a.batch; c.sh = c.gb + a.ng + 1; c.lead = c.sh + a.ng;

  if (tid == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
    mbar_expect_tx(bar, 2 * X::KS);
    bulk_g2s(smem_addr(Ks), a.cbp + cbp_slice_off(g, a.layer, 0, blk, h, step_s), X::KS, bar);
    bulk_g2s(smem_addr(sm + X::OFF_W), a.cbp + cbp_slice_off(g, a.layer, 1, blk, h, step_s), X::KS, bar);
  }
  const bool ok = load_counters(g, a, c, j == 0 && h == 0);   // (its barriers publish the mbarrier)
  // every slot of this part starts empty
  for (int i = tid; i < a.batch * rep * 2; i += kShThreads) {
    const int b = i / (rep * 2), r = i / 2 % rep;
    a.pml[(((size_t)b * g.Hq + h * rep + r) * g.max_splits + j) * 2 + (i & 1)] = make_float2(-INFINITY, 0.f);
  }
  const bool late = __syncthreads_or(!mbar_wait(bar, 0, g.wait_iters));
  if (late || !ok) {
    if (late && tid == 0) {
      set_status(a.st, LVQ_ETIMEOUT);
      mbar_wait(bar, 0, g.wait_iters);                         // the copies land before the CTA exits
    }
    return;
  }
  if (g.pool) check_rows(g, a, c);
  const int n_entries = a.ng + a.batch;
  if (warp == 0) {
    // the cut: costs summed lane by lane
    const int per = (n_entries + 31) / 32;
    long long mine = 0;
    for (int e = lane * per; e < min(n_entries, (lane + 1) * per); ++e) mine += entry_of(g, c, a.ng, e).cost();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) {
      cut[0] = mine * j / a.k;
      cut[1] = mine * (j + 1) / a.k;
    }
  }
  // the slices' largest magnitudes; the values go to their padded rows as scaled fp16
  uint32_t ka = 0, va = 0;
  const uint32_t* kw = reinterpret_cast<const uint32_t*>(Ks);
  const uint32_t* vw = reinterpret_cast<const uint32_t*>(sm + X::OFF_W);
  for (int i = tid; i < X::KS / 4; i += kShThreads) {
    ka = amax_b2(kw[i], ka);
    va = amax_b2(vw[i], va);
  }
  ka = __reduce_max_sync(0xffffffffu, ka);
  va = __reduce_max_sync(0xffffffffu, va);
  if (lane == 0) { red[warp] = ka; red[kWarps + warp] = va; }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) { ka = max(ka, red[w]); va = max(va, red[kWarps + w]); }
  const int kexp = fit_exp(ka), vexp = fit_exp(va) + 1;
  const float vscale = pow2i(vexp), vback = pow2i(-vexp);
  for (int i = tid; i < X::KS / 4; i += kShThreads) {
    const float2 v = b2_lohi(vw[i]);
    *reinterpret_cast<uint32_t*>(Vs + (i / (D / 2)) * X::VROW + (i % (D / 2)) * 4) = pack_h2(v.x * vscale, v.y * vscale);
  }
  // e^{i (S % 8 + j) theta} per lane, and the lane's e^{i 8 theta}
  const float4* rope4 = reinterpret_cast<const float4*>(a.rope);   // two frequencies: (cos, sin, cos, sin)
  auto pair_of = [&](int w) { return ((quad + 4 * (w / (C / 2))) * C + 2 * (w % (C / 2))) / 2; };   // lane's frequency pair w
  if (warp == 0) {
#pragma unroll
    for (int w = 0; w < X::NW; ++w) {
      const int p = (g.S & 7) + row;
      const float4 x = __ldg(rope4 + (size_t)(p >> 3) * (X::F / 2) + pair_of(w));
      const float4 y = __ldg(rope4 + (size_t)(g.RC + (p & 7)) * (X::F / 2) + pair_of(w));
      Ff[w * 32 + lane] = make_float4(x.x * y.x - x.y * y.y, x.z * y.z - x.w * y.w, x.x * y.y + x.y * y.x, x.z * y.w + x.w * y.z);
    }
  }
  float2 ec[X::NW], es[X::NW];
#pragma unroll
  for (int w = 0; w < X::NW; ++w) {
    const float4 x = __ldg(rope4 + X::F / 2 + pair_of(w));
    ec[w] = make_float2(x.x, x.z);
    es[w] = make_float2(x.y, x.w);
  }
  __syncthreads();

  const float qk_scale = 1.4426950408889634f / sqrtf((float)D);
  long long at = 0;
  for (int e = 0; e < n_entries; ++e) {
    const Entry en = entry_of(g, c, a.ng, e);
    if (en.tiles == 0) continue;
    const long long each = kOverhead + en.tiles;
    const int q0 = cut[0] > at ? (int)min((long long)en.qtiles, (cut[0] - at) / each) : 0;
    const long long at0 = at;
    at += en.cost();
    if (at <= cut[0]) continue;
    if (at0 >= cut[1]) break;
    const bool shared = e < a.ng;
    const int lead = shared ? c.lead[e] : e - a.ng;
    for (int qt = q0; qt < en.qtiles; ++qt) {
      const long long base = at0 + qt * each + kOverhead;
      const int t0 = (int)max(0ll, cut[0] - base), t1 = (int)min((long long)en.tiles, cut[1] - base);
      if (base >= cut[1]) break;
      if (t0 >= t1) continue;
      RowTile rt;
      rt.b0 = shared ? c.gb[e] : lead;
      rt.rep = rep; rt.r0 = qt * kQT; rt.h = h;
      rt.nrows = min(kQT, (shared ? (c.gb[e + 1] - c.gb[e]) * rep : rep) - rt.r0);

      // ---- query fragments: D / 4 lanes rotate a row at its own position, scale it to fp16's range and split it
      {
        constexpr int LPR = D / 4, RPW = 32 / LPR;            // lanes of a row, rows a warp takes at once
        const int f2 = lane % LPR;                            // frequency pair
        const int P = 2 * f2 / C, sub = 2 * f2 % C / 2;       // its pair-group and place: fragment lane and k step
        for (int r = warp * RPW + lane / LPR; r < kQT; r += kWarps * RPW) {
          float2 x = make_float2(0.f, 0.f), y = x;
          if (r < rt.nrows && c.ctx[rt.request(r)] > 0) {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q + ((size_t)rt.request(r) * g.Hq + rt.head(r)) * D);
            const int p = c.ctx[rt.request(r)] - 1;
            const float2 q0v = b2_lohi(__ldg(q + f2)), q1v = b2_lohi(__ldg(q + f2 + X::F / 2));
            const float4 u = __ldg(rope4 + (size_t)(p >> 3) * (X::F / 2) + f2);
            const float4 v = __ldg(rope4 + (size_t)(g.RC + (p & 7)) * (X::F / 2) + f2);
            const float c0 = u.x * v.x - u.y * v.y, s0 = u.x * v.y + u.y * v.x;
            const float c1 = u.z * v.z - u.w * v.w, s1 = u.z * v.w + u.w * v.z;
            x = make_float2((q0v.x * c0 - q1v.x * s0) * qk_scale, (q0v.y * c1 - q1v.y * s1) * qk_scale);
            y = make_float2((q1v.x * c0 + q0v.x * s0) * qk_scale, (q1v.y * c1 + q0v.y * s1) * qk_scale);
          }
          float mx = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y)));
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const int qe = mx > 0.f && mx < INFINITY ? min(13 - (((__float_as_int(mx) >> 23) & 255) - 127), 90) : 0;
          const float qs = pow2i(qe);
          uint32_t xh, xl, yh, yl;
          split_h2(make_float2(x.x * qs, x.y * qs), xh, xl);
          split_h2(make_float2(y.x * qs, y.y * qs), yh, yl);
          const int ks = P / 4 * (C / 2) + sub, fl = (r & 7) * 4 + P % 4, rg = r >> 3;
          uint32_t* fh = reinterpret_cast<uint32_t*>(Qf + ks * 32 + fl);
          uint32_t* fw = reinterpret_cast<uint32_t*>(Qf + (X::NW + ks) * 32 + fl);
          fh[rg] = xh; fh[rg + 2] = yh;
          fw[rg] = xl; fw[rg + 2] = yl;
          if (f2 == 0) inv_s[r] = pow2i(-qe);
        }
      }
      __syncthreads();
      uint32_t qh[X::NW][4], ql[X::NW][4];
#pragma unroll
      for (int w = 0; w < X::NW; ++w) {
        const uint4 u = Qf[w * 32 + lane], v = Qf[(X::NW + w) * 32 + lane];
        qh[w][0] = u.x; qh[w][1] = u.y; qh[w][2] = u.z; qh[w][3] = u.w;
        ql[w][0] = v.x; ql[w][1] = v.y; ql[w][2] = v.z; ql[w][3] = v.w;
      }
      const float qinv[2] = {inv_s[row], inv_s[row + 8]};
      State<D, C> st;
#pragma unroll
      for (int i = 0; i < X::NT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) st.o[i][k] = 0.f;
      st.m[0] = st.m[1] = -1e30f;
      st.l[0] = st.l[1] = 0.f;

      // ---- this warp's tiles, by source
      const int w0 = t0 + (int)((long long)(t1 - t0) * warp / kWarps), w1 = t0 + (int)((long long)(t1 - t0) * (warp + 1) / kWarps);
      // source ranges of the entry's tile list: [0, ns) sink, [ns, nc) coded, [nc, tiles) recent
      const int ctx = shared ? 0 : c.ctx[lead];
      const int S_eff = min(g.S, ctx), n_sink_t = ceil_div(S_eff, kTT);
      const int cod0 = shared ? 0 : c.own0[lead], n_cod = shared ? c.sh[e] : c.coded[lead] - cod0;
      const int n_cod_t = n_sink_t + ceil_div(n_cod, kTT);

      // coded tiles
      const int ca = max(w0, n_sink_t), cb = min(w1, n_cod_t);
      if (ca < cb) {
        const uint8_t* kcode = a.idx + idx_page_off(g, a.layer, blk, lead, h, 0, 0);
        const uint8_t* vcode = a.idx + idx_page_off(g, a.layer, blk, lead, h, 1, 0);
        const int pg0 = cod0 / kPage + 2 * (ca - n_sink_t), pg_end = (cod0 + n_cod + kPage - 1) / kPage;
        const float inv[2] = {qinv[0] * pow2i(-kexp), qinv[1] * pow2i(-kexp)};
        int ids = 0, ids_at = -32;                             // physical pages [ids_at, ids_at + 32) of the run, one a lane
        auto fetch = [&](int t) {                              // the codes of run tile t into its stage
          const int pp = 2 * t;
          if (pp - ids_at >= 32) {
            ids_at = pp;
            ids = phys_page(g, lead, min(pg0 + pp + lane, pg_end - 1));
            if (ids < 0) {
              set_status(a.st, LVQ_ECAPACITY);
              ids = 0;
            }
          }
          const int i0 = __shfl_sync(0xffffffffu, ids, pp - ids_at), i1 = __shfl_sync(0xffffffffu, ids, pp + 1 - ids_at);
          const uint32_t dst = smem_addr(area) + (t % X::NST) * X::STAGE;
          constexpr int VP = X::PAGE / 16;
#pragma unroll
          for (int v = lane; v < 4 * VP; v += 32) {
            const int id = (v / VP) & 1 ? i1 : i0;
            cp_async16(dst + v * 16, (v < 2 * VP ? kcode : vcode) + (size_t)id * X::PAGE + v % VP * 16);
          }
        };
        const int nt = cb - ca;
#pragma unroll
        for (int t = 0; t < X::NST - 1; ++t) {
          if (t < nt) fetch(t);
          cp_commit();
        }
        float2 wc[X::NW], ws[X::NW];
        for (int t = 0; t < nt; ++t) {
          cp_wait<X::NST - 2>();
          __syncwarp();
          if (t % 8 == 0) {
            // e^{i p theta} anew from the tables every 16 pages: the recurrence's rounding does not grow further
            const int p8 = pg0 + 2 * t + (g.S >> 3);
            const float ks = pow2i(kexp);
#pragma unroll
            for (int w = 0; w < X::NW; ++w) {
              const float4 x = __ldg(rope4 + (size_t)p8 * (X::F / 2) + pair_of(w));
              const float4 y = Ff[w * 32 + lane];
              wc[w] = make_float2((x.x * y.x - x.y * y.z) * ks, (x.z * y.y - x.w * y.w) * ks);
              ws[w] = make_float2((x.x * y.z + x.y * y.x) * ks, (x.z * y.w + x.w * y.y) * ks);
            }
          }
          const unsigned char* codes = area + (t % X::NST) * X::STAGE;
          float s[2][4] = {};
#pragma unroll
          for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int i = 0; i < X::NI; ++i) {
              const int P = quad + 4 * i;
              const uint32_t k0 = codes[u * X::PAGE + P * kPage + row], k1 = codes[u * X::PAGE + (P + X::NP) * kPage + row];
              const unsigned char* e0 = Ks + k0 * (2 * D) + P * (2 * C);
              const unsigned char* e1 = Ks + k1 * (2 * D) + (P + X::NP) * (2 * C);
#pragma unroll
              for (int q = 0; q < (C + 7) / 8; ++q) {
                uint32_t lo[4], hi[4];
                if constexpr (C == 4) {
                  const uint2 x = *reinterpret_cast<const uint2*>(e0), y = *reinterpret_cast<const uint2*>(e1);
                  lo[0] = x.x; lo[1] = x.y; hi[0] = y.x; hi[1] = y.y;
                } else {
                  const uint4 x = *reinterpret_cast<const uint4*>(e0 + 16 * q), y = *reinterpret_cast<const uint4*>(e1 + 16 * q);
                  lo[0] = x.x; lo[1] = x.y; lo[2] = x.z; lo[3] = x.w;
                  hi[0] = y.x; hi[1] = y.y; hi[2] = y.z; hi[3] = y.w;
                }
#pragma unroll
                for (int v = 0; v < (C < 8 ? C / 2 : 4); ++v) {
                  const int w = i * (C / 2) + q * 4 + v;
                  const float2 ns = neg2(ws[w]);
                  score_pair(s[u], b2_lohi(lo[v]), b2_lohi(hi[v]), wc[w], ws[w], ns, qh[w], ql[w]);
                  const float2 cn = __ffma2_rn(wc[w], ec[w], __fmul2_rn(ns, es[w]));
                  ws[w] = __ffma2_rn(ws[w], ec[w], __fmul2_rn(wc[w], es[w]));
                  wc[w] = cn;
                }
              }
            }
          }
          const int n = min(kTT, n_cod - (ca - n_sink_t + t) * kTT);
          softmax_tile<D, C>(st, s, inv, n, quad);
          uint32_t ph[4], pl[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) split_h2(make_float2(s[k >> 1][2 * (k & 1)], s[k >> 1][2 * (k & 1) + 1]), ph[k], pl[k]);
          // values: channels row * d/8 + 8 q ... of tokens 2 quad, 2 quad + 1 of both pages
          const unsigned char* vc = codes + 2 * X::PAGE + 2 * quad;
          const bool ragged = n < kTT;
#pragma unroll
          for (int q = 0; q < D / 64; ++q) {
            uint32_t v[4][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
              for (int part = 0; part < (C == 4 ? 2 : 1); ++part) {
                const int grp = (row * (D / 8) + 8 * q + 4 * part) / C;
                uint32_t two = *reinterpret_cast<const uint16_t*>(vc + u * X::PAGE + grp * kPage);
                uint32_t c0 = two & 255u, c1 = two >> 8;
                if (ragged) {                                 // masked tokens take the first token's entry: nothing else is read
                  const uint32_t first = codes[2 * X::PAGE + grp * kPage];
                  if (8 * u + 2 * quad >= n) c0 = first;
                  if (8 * u + 2 * quad + 1 >= n) c1 = first;
                }
                const int off = C == 4 ? grp * 8 : (row * (D / 8) + 8 * q) * 2;
                const unsigned char *r0 = Vs + c0 * X::VROW + off, *r1 = Vs + c1 * X::VROW + off;
                if constexpr (C == 4) {
                  const uint2 x = *reinterpret_cast<const uint2*>(r0), y = *reinterpret_cast<const uint2*>(r1);
                  v[2 * u][2 * part] = x.x; v[2 * u][2 * part + 1] = x.y;
                  v[2 * u + 1][2 * part] = y.x; v[2 * u + 1][2 * part + 1] = y.y;
                } else {
                  const uint4 x = *reinterpret_cast<const uint4*>(r0), y = *reinterpret_cast<const uint4*>(r1);
                  v[2 * u][0] = x.x; v[2 * u][1] = x.y; v[2 * u][2] = x.z; v[2 * u][3] = x.w;
                  v[2 * u + 1][0] = y.x; v[2 * u + 1][1] = y.y; v[2 * u + 1][2] = y.z; v[2 * u + 1][3] = y.w;
                }
              }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t sel = i & 1 ? 0x7632u : 0x5410u;
              const uint32_t b0 = __byte_perm(v[0][i >> 1], v[1][i >> 1], sel), b1 = __byte_perm(v[2][i >> 1], v[3][i >> 1], sel);
              mma_f16(st.o[8 * q + i], pl, b0, b1);
              mma_f16(st.o[8 * q + i], ph, b0, b1);
            }
          }
          __syncwarp();                                       // the stage is read
          if (t + X::NST - 1 < nt) fetch(t + X::NST - 1);
          cp_commit();
        }
        cp_wait<0>();
        __syncwarp();
      }

      // bf16 tiles: the sink's, then the recent window's
#pragma unroll 1
      for (int src = 0; src < 2; ++src) {
        const int ra = src == 0 ? w0 : max(w0, n_cod_t), rb = src == 0 ? min(w1, n_sink_t) : w1;
        if (shared) break;
        const int total = src == 0 ? S_eff : ctx - S_eff - c.coded[lead];
#pragma unroll 1
        for (int t = ra; t < rb; ++t) {
          const int i0 = (t - (src == 0 ? 0 : n_cod_t)) * kTT, n = min(kTT, total - i0);
          // rows [K, V][16][d] of the tile; rows that hold no token are zero
          for (int v = lane; v < 2 * kTT * (D / 8); v += 32) {
            const int kv = v / (kTT * (D / 8)), tok = v / (D / 8) % kTT, col = v % (D / 8);
            if (tok < n) {
              const __nv_bfloat16* src_row = src == 0 ? a.sink + sink_off(g, a.layer, kv, a.step, lead, h, i0 + tok)
                                                      : a.ring + ring_off(g, a.layer, kv, a.step, lead, h, (c.coded[lead] + i0 + tok) % g.R);
              cp_async16(smem_addr(area) + v * 16, src_row + col * 8);
            } else {
              *reinterpret_cast<uint4*>(area + v * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          cp_commit();
          cp_wait<0>();
          __syncwarp();
          const int p0 = (src == 0 ? 0 : g.S + c.coded[lead]) + i0 + row;
          float s[2][4] = {};
          uint32_t am = 0;
          for (int v = lane; v < kTT * D / 2; v += 32) am = amax_b2(reinterpret_cast<const uint32_t*>(area)[v], am);
          const int te = fit_exp(__reduce_max_sync(0xffffffffu, am));
          const float ts = pow2i(te);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            // (a row past the last token is zero: its position only has to lie within the tables)
            const int p = min(p0 + 8 * u, g.max_ctx - 1);
#pragma unroll
            for (int w = 0; w < X::NW; ++w) {
              const float4 x = __ldg(rope4 + (size_t)(p >> 3) * (X::F / 2) + pair_of(w));
              const float4 y = __ldg(rope4 + (size_t)(g.RC + (p & 7)) * (X::F / 2) + pair_of(w));
              const float2 cc = make_float2((x.x * y.x - x.y * y.y) * ts, (x.z * y.z - x.w * y.w) * ts);
              const float2 sc = make_float2((x.x * y.y + x.y * y.x) * ts, (x.z * y.w + x.w * y.z) * ts);
              const uint32_t* kr = reinterpret_cast<const uint32_t*>(area) + (8 * u + row) * (D / 2);
              score_pair(s[u], b2_lohi(kr[pair_of(w)]), b2_lohi(kr[pair_of(w) + X::F / 2]), cc, sc, neg2(sc), qh[w], ql[w]);
            }
          }
          const float inv[2] = {qinv[0] * pow2i(-te), qinv[1] * pow2i(-te)};
          softmax_tile<D, C>(st, s, inv, n, quad);
          // bf16 values are exact as they are; the weights as three bf16 parts, in the outputs' scale
          uint32_t pp[3][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float x = s[k >> 1][2 * (k & 1)] * vscale, y = s[k >> 1][2 * (k & 1) + 1] * vscale;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              pp[i][k] = pack_b2(x, y);
              x -= bf16_lo(pp[i][k]);
              y -= bf16_hi(pp[i][k]);
            }
          }
          const uint32_t* vr = reinterpret_cast<const uint32_t*>(area) + kTT * (D / 2) + row * (D / 16);
#pragma unroll
          for (int q = 0; q < X::NT / 2; ++q) {
            const uint32_t x0 = vr[2 * quad * (D / 2) + q], x1 = vr[(2 * quad + 1) * (D / 2) + q];
            const uint32_t y0 = vr[(2 * quad + 8) * (D / 2) + q], y1 = vr[(2 * quad + 9) * (D / 2) + q];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t sel = i ? 0x7632u : 0x5410u;
              const uint32_t b0 = __byte_perm(x0, x1, sel), b1 = __byte_perm(y0, y1, sel);
#pragma unroll
              for (int k = 2; k >= 0; --k) mma_bf16(st.o[2 * q + i], pp[k], b0, b1);
            }
          }
          __syncwarp();
        }
      }

      // ---- the warps' results are joined
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 1);
        st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 2);
        if (quad == 0) ml[warp * kQT + row + 8 * r] = make_float2(st.m[r], st.l[r]);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float* to = reinterpret_cast<float*>(area) + (row + 8 * r) * X::OROW + (2 * quad + n) * X::NT;
#pragma unroll
          for (int i = 0; i < X::NT; i += 4)
            *reinterpret_cast<float4*>(to + i) =
                make_float4(st.o[i][2 * r + n], st.o[i + 1][2 * r + n], st.o[i + 2][2 * r + n], st.o[i + 3][2 * r + n]);
        }
      }
      __syncthreads();
      {
        constexpr int TPR = kShThreads / kQT, CH = D / TPR;   // threads of a row, channels of a thread
        const int r = tid / TPR, c0 = tid % TPR * CH;
        if (r < rt.nrows && c.ctx[rt.request(r)] > 0) {
          float M = -1e30f, L = 0.f, o[CH] = {};
#pragma unroll
          for (int w = 0; w < kWarps; ++w)
            if (ml[w * kQT + r].y > 0.f) M = fmaxf(M, ml[w * kQT + r].x);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 x = ml[w * kQT + r];
            const float f = x.y > 0.f ? ex2(x.x - M) : x.y;   // (a NaN sum stays one)
            L += f * x.y;
            const float* from = reinterpret_cast<const float*>(sm + X::OFF_W + w * X::WARP) + r * X::OROW + c0;
            if (x.y > 0.f || x.y != x.y)
#pragma unroll
              for (int i = 0; i < CH; ++i) o[i] += (x.y > 0.f ? f : x.y) * from[i];
          }
          const size_t slot = (((size_t)rt.request(r) * g.Hq + rt.head(r)) * g.max_splits + j) * 2 + !shared;
#pragma unroll
          for (int i = 0; i < CH; i += 4)
            *reinterpret_cast<float4*>(a.po + slot * D + c0 + i) =
                make_float4(o[i] * vback, o[i + 1] * vback, o[i + 2] * vback, o[i + 3] * vback);
          if (c0 == 0) a.pml[slot] = make_float2(M, L);
        }
      }
      __syncthreads();
    }
  }
}

// Joins the partials of one (request, query head): thread e owns output element e.
template <int D>
__global__ void __launch_bounds__(D) shared_merge_kernel(Geo g, int k, const float* __restrict__ po,
                                                         const float2* __restrict__ pml, float* __restrict__ out,
                                                         float* __restrict__ lse) {
  const int hq = blockIdx.x, b = blockIdx.y, e = threadIdx.x;
  const size_t row = (size_t)b * g.Hq + hq, slot0 = row * g.max_splits * 2;
  float M = -INFINITY;
  for (int i = 0; i < 2 * k; ++i)
    if (pml[slot0 + i].y != 0.f) M = fmaxf(M, pml[slot0 + i].x);
  float den = 0.f, acc = 0.f;
  if (M != -INFINITY)
    for (int i = 0; i < 2 * k; ++i) {
      const float2 ml = pml[slot0 + i];
      if (ml.y != 0.f) {
        const float w = exp2f(ml.x - M);
        den = fmaf(w, ml.y, den);
        acc = fmaf(w, po[(slot0 + i) * D + e], acc);
      }
    }
  out[row * D + e] = den != 0.f ? acc / den : 0.f;
  if (e == 0) lse[row] = den != 0.f ? (M + log2f(den)) * 0.6931471805599453f : -INFINITY;
}

template <int D, int C>
static cudaError_t shared_as(const Geo& g, const SharedArgs& a, float* out, float* lse, cudaStream_t s) {
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
  shared_kernel<D, C><<<dim3(a.k, g.H), kShThreads, Sh<D, C>::smem(a.batch, a.ng), s>>>(g, a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  shared_merge_kernel<D><<<dim3(g.Hq, a.batch), D, 0, s>>>(g, a.k, a.po, a.pml, out, lse);
  return cudaGetLastError();
}

cudaError_t launch_decode_shared(const Geo& g, int layer, int step, int batch, const __nv_bfloat16* q,
                                 const int32_t* ctx_len, const int32_t* coded_len, int n_groups,
                                 const int32_t* group_begin, const int32_t* group_tokens, const __nv_bfloat16* sink,
                                 const __nv_bfloat16* ring, const uint8_t* idx, const __nv_bfloat16* cbp,
                                 const float* rope, int num_splits, float* ws, float* out, float* lse, int32_t* st,
                                 int n_sm, cudaStream_t s) {
  SharedArgs a = {layer, step, batch, n_groups, num_splits, q, ctx_len, coded_len, group_begin, group_tokens,
                  sink, ring, idx, cbp, rope, ws, nullptr, st};
  if (a.k == 0) {
    // one wave of CTAs, but no part below about 128 of the tokens the layout can hold
    const long long most = ((long long)batch * g.max_ctx + 127) / 128;
    a.k = n_sm / g.H < 1 ? 1 : n_sm / g.H;
    if (a.k > g.max_splits) a.k = g.max_splits;
    if (a.k > most) a.k = (int)most;
  }
  a.pml = reinterpret_cast<float2*>(ws + (size_t)g.B * g.Hq * g.max_splits * 2 * g.d);
  if (g.d == 128 && g.c == 4) return shared_as<128, 4>(g, a, out, lse, s);
  if (g.d == 128 && g.c == 8) return shared_as<128, 8>(g, a, out, lse, s);
  if (g.d == 128 && g.c == 16) return shared_as<128, 16>(g, a, out, lse, s);
  if (g.d == 64 && g.c == 4) return shared_as<64, 4>(g, a, out, lse, s);
  if (g.d == 64 && g.c == 8) return shared_as<64, 8>(g, a, out, lse, s);
  return cudaErrorInvalidValue;
}

}  // namespace lvq
