// kv_pool.cu -- which pages of the paged key/value cache belong to which
// sequence (host code only).
//
// A served request decides on the host how long each sequence becomes, so the
// page lists are kept there: allocation, sharing and compaction are a few
// integer operations per page and never wait for the GPU, and their only
// device work is the list of page copies that fork and compact return.
// Free pages are a heap with the lowest number on top, so pages in use stay
// near the front of the pool and the lists depend only on the calls made.
#include <algorithm>
#include <cstdint>
#include <functional>
#include <new>
#include <vector>

#include "../../include/ptl.h"

struct ptl_kv_pool {
  struct Seq {
    std::vector<int32_t> pages;  // -1: given up by trim
    int32_t len = 0;
  };
  std::vector<Seq> seqs;
  std::vector<int32_t> refs;  // sequences that hold the page
  std::vector<int32_t> free_heap;  // capacity num_pages from the start: returning a page cannot fail
  std::vector<uint8_t> mark;  // per sequence, clear between calls

  bool valid(int32_t s) const { return s >= 0 && size_t(s) < seqs.size(); }
  int32_t take() {
    std::pop_heap(free_heap.begin(), free_heap.end(), std::greater<int32_t>());
    const int32_t p = free_heap.back();
    free_heap.pop_back();
    refs[p] = 1;
    return p;
  }
  // returns 1 if the page became free
  int32_t give(int32_t p) {
    if (p < 0 || --refs[p] > 0) return 0;
    free_heap.push_back(p);
    std::push_heap(free_heap.begin(), free_heap.end(), std::greater<int32_t>());
    return 1;
  }
};

namespace {

inline int64_t pages_of(int64_t len) { return (len + PTL_KV_PAGE - 1) / PTL_KV_PAGE; }

// Marks list[0 .. n-1], false at a number out of range or one marked already;
// the marks made are taken back when the guard goes.
struct Marks {
  ptl_kv_pool* pool;
  const int32_t* list;
  int32_t done = 0;
  bool set(int32_t n) {
    for (; done < n; ++done) {
      if (!pool->valid(list[done]) || pool->mark[list[done]]) return false;
      pool->mark[list[done]] = 1;
    }
    return true;
  }
  ~Marks() {
    for (int32_t i = 0; i < done; ++i) pool->mark[list[i]] = 0;
  }
};

}  // namespace

extern "C" {

ptl_status ptl_kv_pool_create(int32_t num_pages, int32_t num_seqs, ptl_kv_pool** pool) {
  if (!pool) return PTL_ERR_NULL;
  *pool = nullptr;
  if (num_pages < 1 || num_seqs < 1) return PTL_ERR_SHAPE;
  ptl_kv_pool* p = nullptr;
  try {
    p = new ptl_kv_pool;
    p->seqs.resize(size_t(num_seqs));
    p->mark.assign(size_t(num_seqs), 0);
    p->refs.assign(size_t(num_pages), 0);
    p->free_heap.resize(size_t(num_pages));
  } catch (...) {
    delete p;
    return PTL_ERR_NO_MEMORY;
  }
  for (int32_t i = 0; i < num_pages; ++i) p->free_heap[i] = i;  // ascending: a heap already
  *pool = p;
  return PTL_OK;
}

void ptl_kv_pool_destroy(ptl_kv_pool* pool) { delete pool; }

ptl_status ptl_kv_pool_reserve(ptl_kv_pool* pool, const int32_t* seqs, const int32_t* new_lens, int32_t n) {
  if (!pool || (n > 0 && (!seqs || !new_lens))) return PTL_ERR_NULL;
  if (n < 0) return PTL_ERR_SHAPE;
  Marks marks{pool, seqs};
  if (!marks.set(n)) return PTL_ERR_SHAPE;
  int64_t need = 0;
  for (int32_t i = 0; i < n; ++i) {
    const ptl_kv_pool::Seq& s = pool->seqs[seqs[i]];
    if (new_lens[i] < s.len) return PTL_ERR_SHAPE;
    need += pages_of(new_lens[i]) - int64_t(s.pages.size());
  }
  if (need > int64_t(pool->free_heap.size())) return PTL_ERR_CACHE_FULL;
  try {
    for (int32_t i = 0; i < n; ++i) {
      std::vector<int32_t>& pages = pool->seqs[seqs[i]].pages;
      const size_t want = size_t(pages_of(new_lens[i]));
      if (want > pages.capacity()) pages.reserve(std::max(want, 2 * pages.capacity()));
    }
  } catch (...) {
    return PTL_ERR_NO_MEMORY;
  }
  for (int32_t i = 0; i < n; ++i) {
    ptl_kv_pool::Seq& s = pool->seqs[seqs[i]];
    while (int64_t(s.pages.size()) < pages_of(new_lens[i])) s.pages.push_back(pool->take());
    s.len = new_lens[i];
  }
  return PTL_OK;
}

ptl_status ptl_kv_pool_fork(ptl_kv_pool* pool, const int32_t* src, const int32_t* dst, int32_t n, int32_t* copy_src,
                            int32_t* copy_dst, int32_t* n_copies) {
  if (!pool || !n_copies || (n > 0 && (!src || !dst || !copy_src || !copy_dst))) return PTL_ERR_NULL;
  if (n < 0) return PTL_ERR_SHAPE;
  Marks marks{pool, dst};
  if (!marks.set(n)) return PTL_ERR_SHAPE;
  int64_t need = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (!pool->valid(src[i]) || pool->mark[src[i]]) return PTL_ERR_SHAPE;
    const ptl_kv_pool::Seq& d = pool->seqs[dst[i]];
    if (d.len != 0 || !d.pages.empty()) return PTL_ERR_SHAPE;
    need += pool->seqs[src[i]].len % PTL_KV_PAGE != 0;
  }
  if (need > int64_t(pool->free_heap.size())) return PTL_ERR_CACHE_FULL;
  try {
    for (int32_t i = 0; i < n; ++i) pool->seqs[dst[i]].pages.reserve(pool->seqs[src[i]].pages.size());
  } catch (...) {
    return PTL_ERR_NO_MEMORY;
  }
  int32_t copies = 0;
  for (int32_t i = 0; i < n; ++i) {
    const ptl_kv_pool::Seq& s = pool->seqs[src[i]];
    ptl_kv_pool::Seq& d = pool->seqs[dst[i]];
    const size_t full = size_t(s.len / PTL_KV_PAGE);
    for (size_t k = 0; k < full; ++k) {
      d.pages.push_back(s.pages[k]);
      if (s.pages[k] >= 0) ++pool->refs[s.pages[k]];
    }
    if (s.len % PTL_KV_PAGE != 0) {
      const int32_t p = pool->take();
      copy_src[copies] = s.pages[full];
      copy_dst[copies++] = p;
      d.pages.push_back(p);
    }
    d.len = s.len;
  }
  *n_copies = copies;
  return PTL_OK;
}

ptl_status ptl_kv_pool_release(ptl_kv_pool* pool, const int32_t* seqs, int32_t n) {
  if (!pool || (n > 0 && !seqs)) return PTL_ERR_NULL;
  if (n < 0) return PTL_ERR_SHAPE;
  for (int32_t i = 0; i < n; ++i)
    if (!pool->valid(seqs[i])) return PTL_ERR_SHAPE;
  for (int32_t i = 0; i < n; ++i) {  // a sequence that appears twice is empty the second time
    ptl_kv_pool::Seq& s = pool->seqs[seqs[i]];
    for (int32_t p : s.pages) pool->give(p);
    s.pages.clear();
    s.len = 0;
  }
  return PTL_OK;
}

ptl_status ptl_kv_pool_trim(ptl_kv_pool* pool, const int32_t* seqs, int32_t n, int32_t window, int32_t sinks,
                            int32_t* freed) {
  if (!pool || (n > 0 && !seqs)) return PTL_ERR_NULL;
  if (n < 0) return PTL_ERR_SHAPE;
  if (window < 1 || sinks < 0) return PTL_ERR_BAD_MASK;
  for (int32_t i = 0; i < n; ++i)
    if (!pool->valid(seqs[i])) return PTL_ERR_SHAPE;
  int32_t count = 0;
  for (int32_t i = 0; i < n; ++i) {
    ptl_kv_pool::Seq& s = pool->seqs[seqs[i]];
    // the next token stands at position len and sees from len - window + 1 on
    const int64_t keep = int64_t(s.len) - window + 1;
    for (size_t k = size_t(pages_of(sinks)); k < s.pages.size() && int64_t(k + 1) * PTL_KV_PAGE <= keep; ++k) {
      if (s.pages[k] < 0) continue;
      count += pool->give(s.pages[k]);
      s.pages[k] = -1;
    }
  }
  if (freed) *freed = count;
  return PTL_OK;
}

ptl_status ptl_kv_pool_compact(ptl_kv_pool* pool, int32_t capacity, int32_t* copy_src, int32_t* copy_dst,
                               int32_t* n_copies) {
  if (!pool || !n_copies || (capacity > 0 && (!copy_src || !copy_dst))) return PTL_ERR_NULL;
  if (capacity < 0) return PTL_ERR_SHAPE;
  const int32_t total = int32_t(pool->refs.size());
  const int32_t used = total - int32_t(pool->free_heap.size());
  int32_t moves = 0;
  for (int32_t p = used; p < total; ++p) moves += pool->refs[p] > 0;
  *n_copies = moves;
  if (moves > capacity) return PTL_ERR_SHAPE;
  if (moves == 0) return PTL_OK;
  std::vector<int32_t> to;
  try {
    to.assign(size_t(total - used), -1);
  } catch (...) {
    return PTL_ERR_NO_MEMORY;
  }
  int32_t hole = 0, i = 0;
  for (int32_t p = used; p < total; ++p) {
    if (pool->refs[p] == 0) continue;
    while (pool->refs[hole] > 0) ++hole;  // as many holes below `used` as pages above
    copy_src[i] = p;
    copy_dst[i++] = hole;
    to[size_t(p - used)] = hole;
    pool->refs[hole] = pool->refs[p];
    pool->refs[p] = 0;
  }
  for (ptl_kv_pool::Seq& s : pool->seqs)
    for (int32_t& p : s.pages)
      if (p >= used) p = to[size_t(p - used)];
  for (int32_t p = used; p < total; ++p) pool->free_heap[size_t(p - used)] = p;  // ascending: a heap
  return PTL_OK;
}

ptl_status ptl_kv_pool_table(const ptl_kv_pool* pool, const int32_t* seqs, int32_t n, int32_t max_pages,
                             int32_t* table) {
  if (!pool || (n > 0 && (!seqs || !table))) return PTL_ERR_NULL;
  if (n < 0 || max_pages < 0) return PTL_ERR_SHAPE;
  for (int32_t i = 0; i < n; ++i)
    if (!pool->valid(seqs[i]) || pool->seqs[seqs[i]].pages.size() > size_t(max_pages)) return PTL_ERR_SHAPE;
  for (int32_t i = 0; i < n; ++i) {
    const std::vector<int32_t>& pages = pool->seqs[seqs[i]].pages;
    int32_t* row = table + int64_t(i) * max_pages;
    std::copy(pages.begin(), pages.end(), row);
    std::fill(row + pages.size(), row + max_pages, -1);
  }
  return PTL_OK;
}

int32_t ptl_kv_pool_length(const ptl_kv_pool* pool, int32_t seq) {
  return pool && pool->valid(seq) ? pool->seqs[seq].len : -1;
}

int32_t ptl_kv_pool_free_pages(const ptl_kv_pool* pool) { return pool ? int32_t(pool->free_heap.size()) : -1; }

}  // extern "C"
