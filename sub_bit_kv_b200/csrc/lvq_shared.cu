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
#include "lvq_common.cuh"

namespace lvq {

namespace {

constexpr int kQT = 16;                 // query rows of a tile
constexpr int kTT = 16;                 // tokens of a tile
constexpr int kOverhead = 4;            // fixed cost of an entry's query tile, in token tiles
constexpr int kShThreads = 256;

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

// e^{i p theta_f} from the coarse (8k) and fine (r < 8) tables
__device__ inline float2 rope_of(const float* rope, int RC, int F, int p, int f) {
  const float2 a = __ldg(reinterpret_cast<const float2*>(rope) + (size_t)(p >> 3) * F + f);
  const float2 b = __ldg(reinterpret_cast<const float2*>(rope) + (size_t)(RC + (p & 7)) * F + f);
  return make_float2(a.x * b.x - a.y * b.y, a.x * b.y + a.y * b.x);
}

// A query tile of an entry: rows r < nrows are (request, query head) pairs.
struct RowTile {
  int b0, rep, r0, nrows, h;
  __device__ int request(int r) const { return b0 + (r0 + r) / rep; }
  __device__ int head(int r) const { return h * rep + (r0 + r) % rep; }
};

}  // namespace

// Token tile t of an entry: 16 consecutive positions from one source.
struct TokenTile {
  int src;          // 0: coded, 1: sink, 2: recent window
  int n0, n;        // first token (coded: of the coded region; sink, recent: of theirs) and tokens used
  int pos;          // position of the first
};
__device__ inline TokenTile token_tile(const Geo& g, const Counters& c, int ng, int e, int t) {
  if (e < ng) return {0, t * kTT, min(kTT, c.sh[e] - t * kTT), g.S + t * kTT};
  const int b = e - ng, ctx = c.ctx[b], S_eff = min(g.S, ctx);
  const int ts = ceil_div(S_eff, kTT);
  if (t < ts) return {1, t * kTT, min(kTT, S_eff - t * kTT), t * kTT};
  t -= ts;
  const int rest = c.coded[b] - c.own0[b], tc = ceil_div(rest, kTT);
  if (t < tc) return {0, c.own0[b] + t * kTT, min(kTT, rest - t * kTT), g.S + c.own0[b] + t * kTT};
  t -= tc;
  const int recent = ctx - S_eff - c.coded[b];
  return {2, t * kTT, min(kTT, recent - t * kTT), g.S + c.coded[b] + t * kTT};
}

template <int D>
__global__ void __launch_bounds__(kShThreads) shared_kernel(Geo g, SharedArgs a) {
  constexpr int F = D / 2, OE = kQT * D / kShThreads;
  extern __shared__ int sm_i[];
  __shared__ float Qs[kQT][D + 1], Ks[kTT][D + 1], Vs[kTT][D], Sc[kQT][kTT + 1], mrow[kQT], lrow[kQT], arow[kQT];
  __shared__ long long cut[2];
  const int tid = threadIdx.x, j = blockIdx.x, h = blockIdx.y, rep = g.Hq / g.H;
  Counters c;
  c.ctx = sm_i; c.coded = c.ctx + a.batch; c.own0 = c.coded + a.batch; c.gb = c.own0 + a.batch; c.sh = c.gb + a.ng + 1; c.lead = c.sh + a.ng;
  const bool ok = load_counters(g, a, c, j == 0 && h == 0);
  // every slot of this part starts empty
  for (int i = tid; i < a.batch * rep * 2; i += kShThreads) {
    const int b = i / (rep * 2), r = i / 2 % rep;
    a.pml[(((size_t)b * g.Hq + h * rep + r) * g.max_splits + j) * 2 + (i & 1)] = make_float2(-INFINITY, 0.f);
  }
  __syncthreads();
  if (!ok) return;
  if (g.pool) check_rows(g, a, c);
  const int n_entries = a.ng + a.batch;
  if (tid == 0) {
    long long W = 0;
    for (int e = 0; e < n_entries; ++e) W += entry_of(g, c, a.ng, e).cost();
    cut[0] = W * j / a.k;
    cut[1] = W * (j + 1) / a.k;
  }
  __syncthreads();
  const int blk = a.step / g.Tc, s = a.step % g.Tc;
  const float scale = 1.4426950408889634f / sqrtf((float)D);
  long long at = 0;
  for (int e = 0; e < n_entries; ++e) {
    const Entry en = entry_of(g, c, a.ng, e);
    for (int qt = 0; en.tiles && qt < en.qtiles; ++qt, at += kOverhead + en.tiles) {
      // token tiles of this query tile that fall into the part
      const int t0 = (int)max(0ll, cut[0] - at - kOverhead), t1 = (int)min((long long)en.tiles, cut[1] - at - kOverhead);
      if (t0 >= t1) continue;
      const bool shared = e < a.ng;
      RowTile rt;
      rt.b0 = shared ? c.gb[e] : e - a.ng;
      rt.rep = rep; rt.r0 = qt * kQT; rt.h = h;
      rt.nrows = min(kQT, (shared ? (c.gb[e + 1] - c.gb[e]) * rep : rep) - rt.r0);
      const int lead = shared ? c.lead[e] : rt.b0;
      for (int i = tid; i < kQT * F; i += kShThreads) {
        const int r = i / F, f = i % F;
        float x = 0.f, y = 0.f;
        if (r < rt.nrows && c.ctx[rt.request(r)] > 0) {
          const __nv_bfloat16* q = a.q + ((size_t)rt.request(r) * g.Hq + rt.head(r)) * D;
          const float q0 = __bfloat162float(q[f]), q1 = __bfloat162float(q[f + F]);
          const float2 w = rope_of(a.rope, g.RC, F, c.ctx[rt.request(r)] - 1, f);
          x = (q0 * w.x - q1 * w.y) * scale;
          y = (q1 * w.x + q0 * w.y) * scale;
        }
        Qs[r][f] = x; Qs[r][f + F] = y;
      }
      if (tid < kQT) { mrow[tid] = -INFINITY; lrow[tid] = 0.f; }
      float o[OE];
      for (int u = 0; u < OE; ++u) o[u] = 0.f;
      const int orow = tid / (kShThreads / kQT), oc = tid % (kShThreads / kQT);
      for (int t = t0; t < t1; ++t) {
        const TokenTile tt = token_tile(g, c, a.ng, e, t);
        __syncthreads();
        for (int i = tid; i < kTT * F; i += kShThreads) {
          const int n = i / F, f = i % F;
          float kx = 0.f, ky = 0.f, vx = 0.f, vy = 0.f;
          if (n < tt.n) {
            const int tok = tt.n0 + n;
            const __nv_bfloat16 *k0, *k1, *v0, *v1;
            if (tt.src == 0) {
              int pg = phys_page(g, lead, tok / kPage);
              if (pg < 0) { set_status(a.st, LVQ_ECAPACITY); pg = 0; }
              const uint8_t* kc = a.idx + idx_page_off(g, a.layer, blk, lead, h, 0, pg) + tok % kPage;
              const uint8_t* vc = a.idx + idx_page_off(g, a.layer, blk, lead, h, 1, pg) + tok % kPage;
              const __nv_bfloat16* kb = a.cbp + cbp_slice_off(g, a.layer, 0, blk, h, s);
              const __nv_bfloat16* vb = a.cbp + cbp_slice_off(g, a.layer, 1, blk, h, s);
              const int g0 = f / g.c, g1 = (f + F) / g.c;
              k0 = kb + kc[g0 * kPage] * D + f; k1 = kb + kc[g1 * kPage] * D + f + F;
              v0 = vb + vc[g0 * kPage] * D + f; v1 = vb + vc[g1 * kPage] * D + f + F;
            } else {
              const __nv_bfloat16* base = tt.src == 1 ? a.sink : a.ring;
              const int row = tt.src == 1 ? tok : (c.coded[lead] + tok) % g.R;
              const size_t ko = tt.src == 1 ? sink_off(g, a.layer, 0, a.step, lead, h, row) : ring_off(g, a.layer, 0, a.step, lead, h, row);
              const size_t vo = tt.src == 1 ? sink_off(g, a.layer, 1, a.step, lead, h, row) : ring_off(g, a.layer, 1, a.step, lead, h, row);
              k0 = base + ko + f; k1 = k0 + F; v0 = base + vo + f; v1 = v0 + F;
            }
            const float2 w = rope_of(a.rope, g.RC, F, tt.pos + n, f);
            const float x = __bfloat162float(*k0), y = __bfloat162float(*k1);
            kx = x * w.x - y * w.y; ky = y * w.x + x * w.y;
            vx = __bfloat162float(*v0); vy = __bfloat162float(*v1);
          }
          Ks[n][f] = kx; Ks[n][f + F] = ky; Vs[n][f] = vx; Vs[n][f + F] = vy;
        }
        __syncthreads();
        {
          const int r = tid / kTT, n = tid % kTT;
          float acc = 0.f;
          for (int f = 0; f < D; ++f) acc = fmaf(Qs[r][f], Ks[n][f], acc);
          Sc[r][n] = n < tt.n ? acc : -INFINITY;
        }
        __syncthreads();
        if (tid < kQT) {
          float m = mrow[tid];
          for (int n = 0; n < tt.n; ++n) m = fmaxf(m, Sc[tid][n]);
          const float al = exp2f(mrow[tid] - m);
          float l = lrow[tid] * al;
          for (int n = 0; n < kTT; ++n) {
            const float p = n < tt.n ? exp2f(Sc[tid][n] - m) : 0.f;
            Sc[tid][n] = p;
            l += p;
          }
          mrow[tid] = m; lrow[tid] = l; arow[tid] = al;
        }
        __syncthreads();
        for (int u = 0; u < OE; ++u) o[u] *= arow[orow];
        for (int n = 0; n < kTT; ++n)
          for (int u = 0; u < OE; ++u) o[u] = fmaf(Sc[orow][n], Vs[n][oc * OE + u], o[u]);
      }
      if (orow < rt.nrows && c.ctx[rt.request(orow)] > 0) {
        const size_t slot = (((size_t)rt.request(orow) * g.Hq + rt.head(orow)) * g.max_splits + j) * 2 + !shared;
        for (int u = 0; u < OE; ++u) a.po[slot * D + oc * OE + u] = o[u];
        if (oc == 0) a.pml[slot] = make_float2(mrow[orow], lrow[orow]);
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
    if (pml[slot0 + i].y > 0.f) M = fmaxf(M, pml[slot0 + i].x);
  float den = 0.f, acc = 0.f;
  if (M != -INFINITY)
    for (int i = 0; i < 2 * k; ++i) {
      const float2 ml = pml[slot0 + i];
      if (ml.y > 0.f) {
        const float w = exp2f(ml.x - M);
        den = fmaf(w, ml.y, den);
        acc = fmaf(w, po[(slot0 + i) * D + e], acc);
      }
    }
  out[row * D + e] = den > 0.f ? acc / den : 0.f;
  if (e == 0) lse[row] = den > 0.f ? (M + log2f(den)) * 0.6931471805599453f : -INFINITY;
}

template <int D>
static cudaError_t shared_as(const Geo& g, const SharedArgs& a, float* out, float* lse, cudaStream_t s) {
  const size_t smem = (size_t)(3 * a.batch + 3 * a.ng + 1) * 4;
  shared_kernel<D><<<dim3(a.k, g.H), kShThreads, smem, s>>>(g, a);
  cudaError_t e = cudaGetLastError();
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
  return g.d == 128 ? shared_as<128>(g, a, out, lse, s) : shared_as<64>(g, a, out, lse, s);
}

}  // namespace lvq
