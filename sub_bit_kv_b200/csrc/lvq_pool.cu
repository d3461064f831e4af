// Host bookkeeping of a page pool (pool mode of lvq_config): which physical page ids are
// handed out to requests, and to how many.  "LoopVQ summary", section "premises and limits": the
// cache is built from 8-token pages; requests of any length take pages from one shared pool as
// their coded region grows and give them back when they end.
//
// Free ids are bits of a map and handed out lowest first, so that the pages of a request tend to
// form runs of consecutive ids, which the decode copies with one bulk copy each.  A page that
// several requests' lists name (forked requests share their parent's full pages, which are never
// written again) has as many holders and is free with the last one.  After lvq_pool_create only
// a renumbering allocates (sets of free and of named ids: 630 us to free 4096 pages, map and stamps: 12).
// Host memory only: the device pools and the page table are the caller's buffers.
#include <algorithm>
#include <new>
#include <vector>

#include "lvq_common.cuh"

struct lvq_pool {
  int32_t n_pages, n_free;
  std::vector<int32_t> holders;     // 0: free
  std::vector<uint64_t> free_map;   // bit id % 64 of word id / 64: id is free
  size_t first;                     // no free id lies in a word before this one
  std::vector<uint32_t> named;      // the last call that named the id (held_once)
  uint32_t call;
};

namespace {

// every id in range, currently handed out, and not repeated
bool held_once(lvq_pool* pool, const int32_t* ids, int32_t n) {
  if (++pool->call == 0) {
    std::fill(pool->named.begin(), pool->named.end(), 0u);
    pool->call = 1;
  }
  for (int32_t i = 0; i < n; ++i) {
    if (ids[i] < 0 || ids[i] >= pool->n_pages || pool->holders[ids[i]] == 0 || pool->named[ids[i]] == pool->call) return false;
    pool->named[ids[i]] = pool->call;
  }
  return true;
}

// The map and its count, from the holders.
void set_free(lvq_pool* pool) {
  std::fill(pool->free_map.begin(), pool->free_map.end(), 0u);
  pool->n_free = 0;
  pool->first = 0;
  for (int32_t i = 0; i < pool->n_pages; ++i)
    if (pool->holders[i] == 0) {
      pool->free_map[i / 64] |= 1ull << i % 64;
      ++pool->n_free;
    }
}

}  // namespace

// No C++ exception (host memory running out) leaves an entry point.
extern "C" {

lvq_status lvq_pool_create(int32_t n_pages, lvq_pool** out) try {
  if (!out || n_pages < 1) return LVQ_EINVAL;
  lvq_pool* p = new (std::nothrow) lvq_pool;
  if (!p) return LVQ_ECAPACITY;
  try {
    p->n_pages = n_pages;
    p->holders.assign(n_pages, 0);
    p->free_map.assign(((size_t)n_pages + 63) / 64, 0);
    p->named.assign(n_pages, 0);
    p->call = 0;
    set_free(p);
  } catch (...) {
    delete p;
    return LVQ_ECAPACITY;
  }
  *out = p;
  return LVQ_OK;
} catch (...) {
  return LVQ_ECAPACITY;
}

void lvq_pool_destroy(lvq_pool* pool) { delete pool; }

lvq_status lvq_pool_alloc(lvq_pool* pool, int32_t n, int32_t* ids) {
  if (!pool || n < 0 || (n > 0 && !ids)) return LVQ_EINVAL;
  if (n > pool->n_free) return LVQ_ECAPACITY;
  for (int32_t i = 0; i < n; ++i) {
    while (pool->free_map[pool->first] == 0) ++pool->first;
    uint64_t& word = pool->free_map[pool->first];
    ids[i] = (int32_t)(pool->first * 64) + __builtin_ctzll(word);
    word &= word - 1;
    pool->holders[ids[i]] = 1;
  }
  pool->n_free -= n;
  return LVQ_OK;
}

lvq_status lvq_pool_share(lvq_pool* pool, const int32_t* ids, int32_t n) {
  if (!pool || n < 0 || (n > 0 && !ids)) return LVQ_EINVAL;
  if (!held_once(pool, ids, n)) return LVQ_EINVAL;
  for (int32_t i = 0; i < n; ++i)
    if (pool->holders[ids[i]] == INT32_MAX) return LVQ_ECAPACITY;
  for (int32_t i = 0; i < n; ++i) ++pool->holders[ids[i]];
  return LVQ_OK;
}

lvq_status lvq_pool_free(lvq_pool* pool, const int32_t* ids, int32_t n) {
  if (!pool || n < 0 || (n > 0 && !ids)) return LVQ_EINVAL;
  if (!held_once(pool, ids, n)) return LVQ_EINVAL;   // all or nothing
  for (int32_t i = 0; i < n; ++i)
    if (--pool->holders[ids[i]] == 0) {
      const size_t word = (size_t)ids[i] / 64;
      pool->free_map[word] |= 1ull << ids[i] % 64;
      pool->first = std::min(pool->first, word);
      ++pool->n_free;
    }
  return LVQ_OK;
}

int32_t lvq_pool_available(const lvq_pool* pool) { return pool ? pool->n_free : -1; }

int32_t lvq_pool_holders(const lvq_pool* pool, int32_t id) {
  return pool && id >= 0 && id < pool->n_pages ? pool->holders[id] : -1;
}

lvq_status lvq_pool_renumber(lvq_pool* pool, const int32_t* new_id) try {
  if (!pool || !new_id) return LVQ_EINVAL;
  const int32_t n = pool->n_pages;
  std::vector<int32_t> holders(n, 0);
  for (int32_t i = 0; i < n; ++i) {
    const int32_t j = new_id[i];
    if (pool->holders[i] == 0) {
      if (j != -1) return LVQ_EINVAL;
      continue;
    }
    if (j < 0 || j >= n || holders[j] != 0) return LVQ_EINVAL;
    holders[j] = pool->holders[i];
  }
  pool->holders.swap(holders);
  set_free(pool);
  return LVQ_OK;
} catch (...) {
  return LVQ_ECAPACITY;
}

// Destination j < m receives page from[j].  The moves form chains that end in a page nobody
// needs any more and cycles.  A chain is listed from its free end (every destination was read
// as an earlier source), so no move reads what an earlier one wrote.  A cycle within one slab
// (reads before writes) is listed as it is; a longer one saves its first destination to
// LVQ_PAGE_HOLD and takes it from there at its end, which then lies in a later slab; a cycle that
// begins in that slab saves only after the slab's reads.
lvq_status lvq_plan_compaction(int32_t n_pages, const int32_t* order, int32_t n_order, int32_t* new_id,
                               int32_t* moves, int32_t* n_moves) try {
  if (n_pages < 1 || n_order < 0 || !new_id || !n_moves || (n_order > 0 && (!order || !moves))) return LVQ_EINVAL;
  if (n_order > (1 << 29)) return LVQ_EUNSUPPORTED;   // (its moves are counted in 32 bits)
  for (int32_t i = 0; i < n_pages; ++i) new_id[i] = -1;
  std::vector<int32_t> from;
  from.reserve(n_order < n_pages ? n_order : n_pages);
  for (int32_t i = 0; i < n_order; ++i) {
    const int32_t id = order[i];
    if (id < 0 || id >= n_pages) return LVQ_EINVAL;
    if (new_id[id] >= 0) continue;
    new_id[id] = (int32_t)from.size();
    from.push_back(id);
  }
  const int32_t m = (int32_t)from.size();
  int32_t k = 0;
  auto emit = [&](int32_t src, int32_t dst) { moves[2 * k] = src; moves[2 * k + 1] = dst; ++k; };
  std::vector<char> done(m, 0);
  for (int32_t j0 = 0; j0 < m; ++j0) {
    if (new_id[j0] >= 0) continue;                 // not the free end of a chain
    for (int32_t j = j0; j < m; j = from[j]) {
      done[j] = 1;
      emit(from[j], j);
    }
  }
  for (int32_t j0 = 0; j0 < m; ++j0) {
    if (done[j0] || from[j0] == j0) continue;
    int32_t len = 0;
    for (int32_t j = j0; !done[j]; j = from[j]) { done[j] = 1; ++len; }
    const bool hold = k % LVQ_MOVE_SLAB + len > LVQ_MOVE_SLAB;
    if (hold) emit(j0, LVQ_PAGE_HOLD);
    int32_t j = j0;
    for (int32_t i = 0; i < len; ++i, j = from[j]) emit(hold && i == len - 1 ? LVQ_PAGE_HOLD : from[j], j);
  }
  *n_moves = k;
  return LVQ_OK;
} catch (...) {
  return LVQ_ECAPACITY;
}

}  // extern "C"
