// Reference counts of a paged cache's pages (vd_pages): allocation, sharing,
// forking and compaction.  Host memory only.
#include <algorithm>
#include <new>
#include <string>
#include <vector>

#include "vd_internal.h"

using vd::fail;

struct vd_pages {
  std::vector<int32_t> refs;
  int32_t free = 0;
};

namespace {

constexpr int32_t kMostRefs = 0x7fffffff;

// A failed allocation of host memory is an error code, not an exception.
template <typename F>
int guarded(F f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return fail(VD_ERR_CAPACITY, "out of host memory");
  }
}

int check_list(const vd_pages* p, int32_t n, const int32_t* pages, bool used) {
  if (!p) return fail(VD_ERR_INVALID_ARG, "null pages");
  if (n < 0) return fail(VD_ERR_INVALID_ARG, "negative number of pages");
  if (n > 0 && !pages) return fail(VD_ERR_INVALID_ARG, "null page list");
  for (int32_t i = 0; i < n; ++i) {
    if (pages[i] < 0 || pages[i] >= static_cast<int32_t>(p->refs.size()))
      return fail(VD_ERR_OUT_OF_RANGE, "page id out of range");
    if (used && p->refs[pages[i]] == 0) return fail(VD_ERR_INVALID_ARG, "page " + std::to_string(pages[i]) + " is free");
  }
  return VD_OK;
}

// `times` more references to each entry, if none overflows.
int retain(vd_pages* p, int32_t n, const int32_t* pages, int32_t times) {
  int32_t i = 0;
  for (; i < n && p->refs[pages[i]] <= kMostRefs - times; ++i) p->refs[pages[i]] += times;
  if (i == n) return VD_OK;
  while (i-- > 0) p->refs[pages[i]] -= times;
  return fail(VD_ERR_CAPACITY, "too many references to a page");
}

void take_lowest(vd_pages* p, int32_t n, int32_t* out) {
  for (int32_t id = 0, k = 0; k < n; ++id)
    if (p->refs[id] == 0) {
      p->refs[id] = 1;
      out[k++] = id;
    }
  p->free -= n;
}

}  // namespace

extern "C" {

int vd_pages_create(int32_t num_pages, vd_pages** out) {
  if (!out) return fail(VD_ERR_INVALID_ARG, "null argument");
  *out = nullptr;
  if (num_pages < 1) return fail(VD_ERR_INVALID_ARG, "num_pages must be >= 1");
  return guarded([&] {
    vd_pages* p = new vd_pages();
    try {
      p->refs.assign(num_pages, 0);
    } catch (...) {
      delete p;
      throw;
    }
    p->free = num_pages;
    *out = p;
    return VD_OK;
  });
}

void vd_destroy_pages(vd_pages* p) { delete p; }

int32_t vd_pages_free(const vd_pages* p) { return p ? p->free : -1; }

int32_t vd_pages_refs(const vd_pages* p, int32_t page) {
  return p && page >= 0 && page < static_cast<int32_t>(p->refs.size()) ? p->refs[page] : -1;
}

int vd_pages_alloc(vd_pages* p, int32_t n, int32_t* out) {
  if (!p) return fail(VD_ERR_INVALID_ARG, "null pages");
  if (n < 0) return fail(VD_ERR_INVALID_ARG, "negative number of pages");
  if (n > 0 && !out) return fail(VD_ERR_INVALID_ARG, "null page list");
  if (n > p->free) return fail(VD_ERR_CAPACITY, "too few free pages");
  take_lowest(p, n, out);
  return VD_OK;
}

int vd_pages_retain(vd_pages* p, int32_t n, const int32_t* pages) {
  if (const int rc = check_list(p, n, pages, true)) return rc;
  return retain(p, n, pages, 1);
}

int vd_pages_release(vd_pages* p, int32_t n, const int32_t* pages) {
  if (const int rc = check_list(p, n, pages, true)) return rc;
  for (int32_t i = 0; i < n; ++i) {
    if (p->refs[pages[i]] == 0) {  // listed more often than referenced: as before
      const std::string id = std::to_string(pages[i]);
      while (i-- > 0) p->free -= p->refs[pages[i]]++ == 0;
      return fail(VD_ERR_INVALID_ARG, "page " + id + " is released more often than it is referenced");
    }
    p->free += --p->refs[pages[i]] == 0;
  }
  return VD_OK;
}

int vd_pages_fork(vd_pages* p, int32_t n, int32_t n_shared, const int32_t* table, int32_t children, int32_t* out,
                  int32_t* src, int32_t* dst) {
  if (const int rc = check_list(p, n, table, true)) return rc;
  if (n_shared < 0 || n_shared > n || children < 0)
    return fail(VD_ERR_INVALID_ARG, "0 <= n_shared <= n and children >= 0 are needed");
  const int32_t own = n - n_shared;
  if (n == 0 || children == 0) return VD_OK;
  if (!out || (own > 0 && (!src || !dst))) return fail(VD_ERR_INVALID_ARG, "null argument");
  if (static_cast<long long>(own) * children > p->free) return fail(VD_ERR_CAPACITY, "too few free pages");
  if (const int rc = retain(p, n_shared, table, children)) return rc;
  if (own > 0) take_lowest(p, own * children, dst);
  for (int32_t k = 0; k < children; ++k)
    for (int32_t j = 0; j < n; ++j) {
      int32_t& to = out[static_cast<size_t>(k) * n + j];
      if (j < n_shared) {
        to = table[j];
      } else {
        const size_t i = static_cast<size_t>(k) * own + (j - n_shared);
        src[i] = table[j];
        to = dst[i];
      }
    }
  return VD_OK;
}

int vd_pages_compact(vd_pages* p, int32_t max_moves, int32_t* src, int32_t* dst, int32_t* n_moves, int32_t n_entries,
                     int32_t* tables) {
  if (!p || !n_moves) return fail(VD_ERR_INVALID_ARG, "null argument");
  if (max_moves < 0 || n_entries < 0) return fail(VD_ERR_INVALID_ARG, "negative size");
  if ((max_moves > 0 && (!src || !dst)) || (n_entries > 0 && !tables)) return fail(VD_ERR_INVALID_ARG, "null argument");
  const int32_t N = static_cast<int32_t>(p->refs.size());
  for (int32_t i = 0; i < n_entries; ++i) {
    if (tables[i] >= N) return fail(VD_ERR_OUT_OF_RANGE, "page id out of range");
    if (tables[i] >= 0 && p->refs[tables[i]] == 0)
      return fail(VD_ERR_INVALID_ARG, "page " + std::to_string(tables[i]) + " is free");
  }
  return guarded([&] {
    std::vector<int32_t> to(N, -1);
    int32_t lo = 0, hi = N - 1, k = 0;
    while (k < max_moves) {
      while (lo < N && p->refs[lo] > 0) ++lo;
      while (hi >= 0 && p->refs[hi] == 0) --hi;
      if (lo >= hi) break;
      src[k] = hi;
      dst[k++] = lo;
      to[hi] = lo;
      std::swap(p->refs[lo], p->refs[hi]);
    }
    for (int32_t i = 0; i < n_entries; ++i)
      if (tables[i] >= 0 && to[tables[i]] >= 0) tables[i] = to[tables[i]];
    *n_moves = k;
    return VD_OK;
  });
}

}  // extern "C"
