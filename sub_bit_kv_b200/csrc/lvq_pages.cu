// Pages and requests moved on the device: copying pages, compacting the pool, forking requests.
// "LoopVQ summary", section "premises and limits": the cache is built from 8-token pages, one
// index row per block of loop steps.  A physical page id means the same place in every (layer,
// block, head, K/V) pool, so moving one page moves page_bytes (64 to 256) in each of them.
//
// No arithmetic: all three are bound by HBM, one read of what is copied and one write of each copy.
#include "lvq_common.cuh"

namespace lvq {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;                         // 16-byte loads in flight per thread
constexpr int kTile = kThreads * kUnroll;          // vectors of one tile

__device__ inline uint4 load16(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

__device__ inline bool in_pool(const Geo& g, int id) { return id >= 0 && id < g.pool; }

}  // namespace

// ---------------------------------------------------------------------------- copy

// Pair (src, dst) in every stream: grid (tiles over the pairs' 16-byte vectors, streams).  The
// pairs have no order, so every vector is a thread of its own.
__global__ void __launch_bounds__(kThreads) copy_pages_kernel(Geo g, int n, int n_streams,
                                                              const int2* __restrict__ pairs, uint8_t* idx,
                                                              int32_t* st) {
  const int vpp = g.page_bytes / 16;               // 4, 8 or 16 vectors a page
  const int lg = __ffs(vpp) - 1;
  const size_t stream_bytes = (size_t)g.pool * g.page_bytes;
  const long long total = (long long)n << lg;
  for (int s = blockIdx.y; s < n_streams; s += gridDim.y) {
    uint8_t* base = idx + (size_t)s * stream_bytes;
    for (long long t0 = (long long)blockIdx.x * kTile; t0 < total; t0 += (long long)gridDim.x * kTile) {
      uint4 v[kUnroll];
      uint4* to[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const long long i = t0 + u * kThreads + threadIdx.x;
        to[u] = nullptr;
        if (i >= total) continue;
        const int2 p = __ldg(pairs + (i >> lg));
        if (!in_pool(g, p.x) || !in_pool(g, p.y)) {
          set_status(st, LVQ_ECAPACITY);
          continue;
        }
        const int col = (int)(i & (vpp - 1)) * 16;
        v[u] = load16(reinterpret_cast<const uint4*>(base + (size_t)p.x * g.page_bytes + col));
        to[u] = reinterpret_cast<uint4*>(base + (size_t)p.y * g.page_bytes + col);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (to[u]) *to[u] = v[u];
    }
  }
}

cudaError_t launch_copy_pages(const Geo& g, int n, const int32_t* pairs, uint8_t* idx, int32_t* st, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const int n_streams = g.L * g.nblk * g.H * 2;
  const long long tiles = ((long long)n * (g.page_bytes / 16) + kTile - 1) / kTile;
  const dim3 grid((unsigned)(tiles < (1 << 20) ? tiles : (1 << 20)), n_streams < 65535 ? n_streams : 65535);
  copy_pages_kernel<<<grid, kThreads, 0, s>>>(g, n, n_streams, reinterpret_cast<const int2*>(pairs), idx, st);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------- compaction

// Moves in list order, slab by slab: one CTA owns CW vectors of every page of one stream (the
// columns of a page and the streams do not depend on one another), reads a slab's sources into
// registers and, behind a barrier, writes its destinations.  No read needs a value that an
// earlier slab wrote (chains are listed from their free end), except through the hold page, which
// lives in shared memory and is read only when the slab is written; so the next slab's reads are
// issued before this slab's writes, and the list streams at full memory parallelism.
// CTAs past the last stream rewrite the page table.
template <int CW>
__global__ void __launch_bounds__(kThreads, 6) compact_pages_kernel(Geo g, int n_moves, int n_move_ctas,
                                                                    const int2* __restrict__ moves,
                                                                    const int32_t* __restrict__ new_id,
                                                                    int32_t* table, uint8_t* idx, int32_t* st) {
  constexpr int U = LVQ_MOVE_SLAB * CW / kThreads;   // vectors of a slab per thread
  constexpr int PT = kThreads / CW;                  // pages one round of the block's threads covers
  static_assert(U >= 1 && U * PT == LVQ_MOVE_SLAB, "slab mapping");
  const int tid = threadIdx.x;
  if ((int)blockIdx.x >= n_move_ctas) {
    const long long total = (long long)g.B * g.pts;
    for (long long i = (long long)(blockIdx.x - n_move_ctas) * kThreads + tid; i < total;
         i += (long long)(gridDim.x - n_move_ctas) * kThreads) {
      const int id = table[i];
      if (in_pool(g, id)) {
        const int to = __ldg(new_id + id);
        table[i] = in_pool(g, to) ? to : -1;
      }
    }
    return;
  }
  __shared__ uint4 hold[CW];
  const int groups = g.page_bytes / 16 / CW;         // column groups of a page
  const size_t stream = blockIdx.x / groups;
  const int col = tid % CW;
  uint4* base = reinterpret_cast<uint4*>(idx + stream * (size_t)g.pool * g.page_bytes) + (blockIdx.x % groups) * CW + col;
  const size_t vpp = g.page_bytes / 16;
  const int p0 = tid / CW;

  // the moves are fetched two slabs ahead, the pages one
  int2 mv[U], mn[U], mf[U];
  uint4 v[U], vn[U];
  auto fetch = [&](int s0, int2 (&m)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = s0 + p0 + u * PT;
      m[u] = i < n_moves ? __ldg(moves + i) : make_int2(-2, -2);
    }
  };
  auto load = [&](int s0, int2 (&m)[U], uint4 (&x)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if ((m[u].x != LVQ_PAGE_HOLD && !in_pool(g, m[u].x)) || (m[u].y != LVQ_PAGE_HOLD && !in_pool(g, m[u].y))) {
        if (s0 + p0 + u * PT < n_moves) set_status(st, LVQ_ECAPACITY);
        m[u] = make_int2(-2, -2);
      }
      if (m[u].x >= 0) x[u] = load16(base + (size_t)m[u].x * vpp);
    }
  };
  fetch(0, mv);
  fetch(LVQ_MOVE_SLAB, mn);
  load(0, mv, v);
  for (int s0 = 0; s0 < n_moves; s0 += LVQ_MOVE_SLAB) {
    fetch(s0 + 2 * LVQ_MOVE_SLAB, mf);
    load(s0 + LVQ_MOVE_SLAB, mn, vn);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (mv[u].x == LVQ_PAGE_HOLD) v[u] = hold[col];
    __syncthreads();                                 // every read of this slab (and the next) precedes its writes
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (mv[u].y >= 0) base[(size_t)mv[u].y * vpp] = v[u];
      if (mv[u].y == LVQ_PAGE_HOLD) hold[col] = v[u];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) { mv[u] = mn[u]; v[u] = vn[u]; mn[u] = mf[u]; }
  }
}

cudaError_t launch_compact_pages(const Geo& g, int n_moves, const int32_t* moves, const int32_t* new_id, int32_t* table,
                                 uint8_t* idx, int32_t* st, int n_sm, cudaStream_t s) {
  const long long streams = (long long)g.L * g.nblk * g.H * 2;
  const int vpp = g.page_bytes / 16;
  // few streams: a page's columns are spread over more CTAs, down to 64-byte pieces
  const int cw = vpp >= 8 && streams * (vpp / 8) >= 2 * n_sm ? 8 : 4;
  const long long move_ctas = n_moves > 0 ? streams * (vpp / cw) : 0;
  const long long entries = (long long)g.B * g.pts;
  const long long table_ctas = (entries + kTile - 1) / kTile < 1024 ? (entries + kTile - 1) / kTile : 1024;
  if (move_ctas + table_ctas > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)(move_ctas + table_ctas);
  const int2* mv = reinterpret_cast<const int2*>(moves);
  if (cw == 8) compact_pages_kernel<8><<<grid, kThreads, 0, s>>>(g, n_moves, (int)move_ctas, mv, new_id, table, idx, st);
  else compact_pages_kernel<4><<<grid, kThreads, 0, s>>>(g, n_moves, (int)move_ctas, mv, new_id, table, idx, st);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------- fork

// CTAs by what they copy, in this order; every one reads its part of the parent once and writes it
// to each child.
struct ForkPlan {
  long long ring_ctas, sink_ctas, code_ctas, row_ctas;   // row_ctas: one per child (page-table row, counters)
  int ring_tiles, sink_tiles, code_tiles;                // tiles of one (layer, K/V, step) or code stream
  int n, parent, coded;
  int child[kForkMax], tail[kForkMax];                   // tail: the child's copy of the partial page, -1 without one
};

__global__ void __launch_bounds__(kThreads) fork_kernel(Geo g, const __grid_constant__ ForkPlan f, int32_t* ctx_len,
                                                        int32_t* coded_len, uint4* sink, uint4* ring, uint8_t* idx,
                                                        int32_t* table, int32_t* st) {
  const int tid = threadIdx.x;
  const int ctx = ctx_len[f.parent], coded = coded_len[f.parent];
  const int S_eff = min(g.S, max(ctx, 0)), recent = ctx - S_eff - coded;
  const bool outside = ctx < 1 || ctx > g.max_ctx || coded < 0 || coded > g.P * kPage || (coded > 0 && ctx < g.S + coded) ||
                       recent < 0 || recent > g.R;
  if (coded != f.coded || outside) {
    if (tid == 0) set_status(st, coded != f.coded ? LVQ_EINVAL : LVQ_ECAPACITY);
    return;
  }
  const int full = coded / kPage;
  int tail_src = -1;
  if (g.pool && coded % kPage) {
    tail_src = phys_page(g, f.parent, full);
    if (tail_src < 0) {
      if (tid == 0) set_status(st, LVQ_ECAPACITY);
      return;
    }
  }
  const int vpr = g.d / 8;                                // 16-byte vectors of a bf16 row
  long long c = blockIdx.x;
  if (c < f.ring_ctas || c < f.ring_ctas + f.sink_ctas) {
    // sink rows or ring rows of one (layer, K/V, step): [B][H][rows][d]
    const bool is_ring = c < f.ring_ctas;
    if (!is_ring) c -= f.ring_ctas;
    const int tiles = is_ring ? f.ring_tiles : f.sink_tiles, rows = is_ring ? g.R : g.S;
    const size_t per_req = (size_t)g.H * rows * vpr;
    uint4* unit = (is_ring ? ring : sink) + (size_t)(c / tiles) * g.B * per_req;
    const uint4* from = unit + f.parent * per_req;
    const unsigned i0 = (unsigned)(c % tiles) * kTile + tid;
    const int oldest = coded % g.R;
    uint4 v[kUnroll];
    bool live[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const unsigned i = i0 + u * kThreads;
      const int row = (int)((i / vpr) % (unsigned)rows);
      int age = row - oldest;                             // slot of the ring -> place among the recent tokens
      if (age < 0) age += g.R;
      live[u] = i < per_req && (is_ring ? age < recent : row < S_eff);
      if (live[u]) v[u] = load16(from + i);
    }
    for (int k = 0; k < f.n; ++k) {
      uint4* to = unit + f.child[k] * per_req;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (live[u]) to[i0 + u * kThreads] = v[u];
    }
    return;
  }
  c -= f.ring_ctas + f.sink_ctas;
  if (c < f.code_ctas) {
    if (g.pool) {
      // the partial page of every stream
      const int vpp = g.page_bytes / 16;
      const long long i = c * kThreads + tid;
      const long long stream = i / vpp;
      if (tail_src < 0 || stream >= (long long)g.L * g.nblk * g.H * 2) return;
      uint4* base = reinterpret_cast<uint4*>(idx + (size_t)stream * g.pool * g.page_bytes) + i % vpp;
      const uint4 v = load16(base + (size_t)tail_src * vpp);
      for (int k = 0; k < f.n; ++k)
        if (f.tail[k] >= 0) base[(size_t)f.tail[k] * vpp] = v;
    } else {
      // the code pages of one (layer, block, head, K/V): [layer][block][B][H * 2][page]
      const long long unit = c / f.code_tiles;
      const size_t stream = (size_t)g.P * g.page_bytes / 16, hs = (size_t)g.H * 2;
      uint4* base = reinterpret_cast<uint4*>(idx) + ((unit / hs) * g.B * hs + unit % hs) * stream;
      const size_t n_vec = (size_t)((coded + kPage - 1) / kPage) * g.page_bytes / 16;
      const size_t i0 = (size_t)(c % f.code_tiles) * kTile + tid;
      uint4 v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (i0 + u * kThreads < n_vec) v[u] = load16(base + f.parent * hs * stream + i0 + u * kThreads);
      for (int k = 0; k < f.n; ++k)
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (i0 + u * kThreads < n_vec) base[f.child[k] * hs * stream + i0 + u * kThreads] = v[u];
    }
    return;
  }
  const int k = (int)(c - f.code_ctas);
  const int b = f.child[k];
  if (g.pool) {
    const int32_t* src = table + (size_t)f.parent * g.pts;
    int32_t* dst = table + (size_t)b * g.pts;
    for (int i = tid; i < g.pts; i += kThreads) dst[i] = i < full ? src[i] : i == full && coded % kPage ? f.tail[k] : -1;
  }
  if (tid == 0) {
    ctx_len[b] = ctx;
    coded_len[b] = coded;
  }
}

cudaError_t launch_fork(const Geo& g, int parent, int n, const int32_t* children, int coded, const int32_t* tails,
                        int32_t* ctx_len, int32_t* coded_len, __nv_bfloat16* sink, __nv_bfloat16* ring, uint8_t* idx,
                        int32_t* table, int32_t* st, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  ForkPlan f = {};
  f.n = n; f.parent = parent; f.coded = coded;
  for (int k = 0; k < n; ++k) {
    f.child[k] = children[k];
    f.tail[k] = tails ? tails[k] : -1;
  }
  const long long units = (long long)g.L * 2 * g.T, streams = (long long)g.L * g.nblk * g.H * 2;
  auto tiles = [](long long v) { return (v + kTile - 1) / kTile; };
  const long long rt = tiles((long long)g.H * g.R * (g.d / 8)), sk = tiles((long long)g.H * g.S * (g.d / 8));
  if (rt * kTile > INT32_MAX || sk * kTile > INT32_MAX) return cudaErrorInvalidValue;   // 32-bit places in a unit
  f.ring_tiles = (int)rt; f.sink_tiles = (int)sk;
  f.ring_ctas = units * rt; f.sink_ctas = units * sk;
  if (g.pool) {
    f.code_ctas = coded % kPage ? (streams * (g.page_bytes / 16) + kThreads - 1) / kThreads : 0;
  } else {
    f.code_tiles = (int)tiles((long long)((coded + kPage - 1) / kPage) * g.page_bytes / 16);
    f.code_ctas = streams * f.code_tiles;
  }
  f.row_ctas = n;
  const long long grid = f.ring_ctas + f.sink_ctas + f.code_ctas + f.row_ctas;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  fork_kernel<<<(unsigned)grid, kThreads, 0, s>>>(g, f, ctx_len, coded_len, reinterpret_cast<uint4*>(sink),
                                                  reinterpret_cast<uint4*>(ring), idx, table, st);
  return cudaGetLastError();
}

}  // namespace lvq
