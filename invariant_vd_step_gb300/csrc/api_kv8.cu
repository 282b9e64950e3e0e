// C ABI of the 8-bit KV cache (vd_kv8): the cache, plans of steps over it, the
// ops of a layer and the whole step, and page copies.
#include <math.h>

#include <algorithm>
#include <atomic>
#include <new>
#include <string>
#include <unordered_set>
#include <utility>
#include <vector>

#include "vd_internal.h"
#include "vd_model.h"

using namespace vd;

struct vd_kv8 {
  vd_model* m = nullptr;
  unsigned long long id = 0;  // never reused, unlike the host address
  int device = 0, format = 0, num_pages = 0;
  void* data = nullptr;
  bool owned = false;
  uint8_t* codes(int layer) const { return static_cast<uint8_t*>(data) + layer * codes_layer(); }
  float4* scales(int layer) const {
    return reinterpret_cast<float4*>(static_cast<uint8_t*>(data) + m->cfg.n_layers * codes_layer()) +
           layer * scales_layer();
  }
  long long codes_layer() const { return static_cast<long long>(num_pages) * m->cfg.n_kv_heads * 32 * m->cfg.head_dim; }
  long long scales_layer() const { return static_cast<long long>(num_pages) * m->cfg.n_kv_heads; }
};

struct vd_kv8_plan {
  vd_model* m = nullptr;
  int device = 0, max_tokens = 0;
  int prefill = 0;  // vd_kv8_set_prefill
  // the plan in force
  Desc d;
  unsigned long long pool_id = 0, cache_id = 0;
  bool planned = false, has_tokens = false;
  // device copy of the plan and split partials; both grow with the plans
  int* dev = nullptr;
  size_t dev_cap = 0;  // ints
  float* part = nullptr;
  size_t part_cap = 0;  // floats
  uint8_t* images = nullptr;
  size_t images_cap = 0;
  int* host[2] = {nullptr, nullptr};  // pinned staging
  size_t host_cap[2] = {0, 0};
  cudaEvent_t uploaded[2] = {nullptr, nullptr};
  int slot = 0;
};

namespace {

constexpr int kSplitPages = kAttn8Split / 16;
// Images that the choice of kernels may ask for: 65 KB for 128 keys of a KV head of 128
// dims, twice the bytes of the same keys' codes in one layer, so histories of 16 M such
// keys (2 M tokens of 8 heads).  Chunks beyond them go to mma.sync.
constexpr size_t kMostImageBytes = static_cast<size_t>(8) << 30;

int check_device(const vd_model* m) {
  int dev = -1;
  VD_CUDA_TRY(cudaGetDevice(&dev));
  if (dev != m->device) return fail(VD_ERR_INVALID_ARG, "the model lives on another device than the current one");
  return VD_OK;
}

int check_pair(const vd_kv8* c, const vd_kv_pool* pool) {
  if (!c || !pool) return fail(VD_ERR_INVALID_ARG, "null cache or pool");
  if (pool->m != c->m) return fail(VD_ERR_INVALID_ARG, "the pool belongs to another model than the cache");
  return check_device(c->m);
}

int check_call(const vd_kv8_plan* p, const vd_kv8* c, const vd_kv_pool* pool, cudaStream_t s) {
  if (!p || !c || !pool) return fail(VD_ERR_INVALID_ARG, "null plan, cache or pool");
  if (c->m != p->m || pool->m != p->m) return fail(VD_ERR_INVALID_ARG, "the cache or pool belongs to another model");
  if (const int rc = check_device(p->m)) return rc;
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  VD_CUDA_TRY(cudaStreamIsCapturing(s, &cap));
  if (cap != cudaStreamCaptureStatusNone)
    return fail(VD_ERR_UNSUPPORTED, "calls on a plan cannot be captured: it changes from step to step");
  return VD_OK;
}

int check_planned(const vd_kv8_plan* p, const vd_kv8* c, const vd_kv_pool* pool, cudaStream_t s) {
  if (const int rc = check_call(p, c, pool, s)) return rc;
  if (!p->planned) return fail(VD_ERR_INVALID_ARG, "nothing has been planned");
  if (p->pool_id != pool->id || p->cache_id != c->id)
    return fail(VD_ERR_INVALID_ARG, "the step was planned for another cache or pool");
  return VD_OK;
}

int check_layer(const vd_model* m, int layer) {
  return layer < 0 || layer >= m->cfg.n_layers ? fail(VD_ERR_OUT_OF_RANGE, "layer out of range") : VD_OK;
}

// Page ids of a copy-like call.  `across`: src and dst are pages of one space.
int check_pages(int n, const int* src, const int* dst, int src_pages, int dst_pages, bool across) {
  if (n < 0) return fail(VD_ERR_INVALID_ARG, "negative number of pages");
  if (n > 0 && (!src || !dst)) return fail(VD_ERR_INVALID_ARG, "null page list");
  for (int i = 0; i < n; ++i)
    if (src[i] < 0 || src[i] >= src_pages || dst[i] < 0 || dst[i] >= dst_pages)
      return fail(VD_ERR_OUT_OF_RANGE, "page id out of range");
  // A mark per page, or for few pages of many the sorted list: 3 of a million 0.04 us
  // instead of 28, 448 of a million 10.5 instead of 27, 448 of 65536 9.6 where the
  // marks take 1.5.
  if (n < dst_pages / 2048) {
    std::vector<int> sorted(dst, dst + n);
    std::sort(sorted.begin(), sorted.end());
    if (std::adjacent_find(sorted.begin(), sorted.end()) != sorted.end())
      return fail(VD_ERR_INVALID_ARG, "a page is written twice");
    for (int i = 0; across && i < n; ++i)
      if (std::binary_search(sorted.begin(), sorted.end(), src[i]))
        return fail(VD_ERR_INVALID_ARG, "a page is both a source and a destination");
    return VD_OK;
  }
  std::vector<unsigned char> seen(n > 0 ? dst_pages : 0, 0);
  for (int i = 0; i < n; ++i) {
    if (seen[dst[i]]) return fail(VD_ERR_INVALID_ARG, "a page is written twice");
    seen[dst[i]] = 1;
  }
  if (across)
    for (int i = 0; i < n; ++i)
      if (seen[src[i]]) return fail(VD_ERR_INVALID_ARG, "a page is both a source and a destination");
  return VD_OK;
}

template <typename P, typename F>
int for_pairs_of(int n, const int* src, const int* dst, F launch) {
  for (int i = 0; i < n; i += P::kMost) {
    P p;
    p.dev = nullptr;
    p.n = std::min(P::kMost, n - i);
    for (int k = 0; k < p.n; ++k) p.at[k] = make_int2(src[i + k], dst[i + k]);
    if (const int rc = launch(p)) return rc;
  }
  return VD_OK;
}
template <typename F>
int for_pairs(int n, const int* src, const int* dst, F launch) {
  return n <= PagePairs::kMost ? for_pairs_of<PagePairs>(n, src, dst, launch) : for_pairs_of<ManyPagePairs>(n, src, dst, launch);
}

SealArgs seal_args(const vd_kv8* c, const vd_kv_pool* pool, int layer) {  // layer -1: all
  const vd_model_config& f = c->m->cfg;
  SealArgs a{};
  a.pool_layer = static_cast<long long>(pool->num_pages) * 2 * f.n_kv_heads * 16 * f.head_dim;
  a.codes_layer = c->codes_layer();
  a.scales_layer = c->scales_layer();
  const int l0 = std::max(layer, 0);
  a.pool = static_cast<__nv_bfloat16*>(pool->data) + l0 * a.pool_layer;
  a.codes = c->codes(l0);
  a.scales = c->scales(l0);
  a.layers = layer < 0 ? f.n_layers : 1;
  a.Hkv = f.n_kv_heads;
  a.hd = f.head_dim;
  a.format = c->format;
  return a;
}

int seal_call(vd_kv8* c, vd_kv_pool* pool, int layer, int n, const int* src, const int* dst, bool unseal, void* stream) {
  if (const int rc = check_pair(c, pool)) return rc;
  if (layer < -1 || layer >= c->m->cfg.n_layers) return fail(VD_ERR_OUT_OF_RANGE, "layer out of range");
  const int np = pool->num_pages, nc = c->num_pages;
  if (const int rc = check_pages(n, src, dst, unseal ? nc : np, unseal ? np : nc, false)) return rc;
  const SealArgs a = seal_args(c, pool, layer);
  return for_pairs(n, src, dst, [&](const auto& p) {
    return launch_kv8_seal(a, p, unseal, static_cast<cudaStream_t>(stream));
  });
}

// Grows a device buffer to at least n elements (the old one is freed once the
// device is done with it), by half of it for the plans to come, 64 MB at most, where
// there is room for that.
template <typename T>
int grow(T** p, size_t* cap, size_t n) {
  if (n <= *cap) return VD_OK;
  size_t want = std::max(n, *cap + std::min(*cap / 2, (static_cast<size_t>(64) << 20) / sizeof(T)));
  if (*p) cudaFree(*p);
  *p = nullptr;
  *cap = 0;
  if (want > n && cudaMalloc(reinterpret_cast<void**>(p), want * sizeof(T)) != cudaSuccess) {
    cudaGetLastError();  // (the error is this attempt's)
    *p = nullptr;
    want = n;
  }
  if (!*p) VD_CUDA_TRY(cudaMalloc(reinterpret_cast<void**>(p), want * sizeof(T)));
  *cap = want;
  return VD_OK;
}

// A call's host containers may fail to allocate; no exception leaves the C ABI.
template <typename F>
int guarded(F f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return fail(VD_ERR_CAPACITY, "out of host memory");
  }
}

int make_plan(vd_kv8_plan* t, vd_kv8* cache, vd_kv_pool* pool, const vd_kv8_batch* b, cudaStream_t s) {
  vd_model* m = t->m;
  const vd_model_config& c = m->cfg;
  if (!b) return fail(VD_ERR_INVALID_ARG, "null batch");
  const int T = b->num_tokens, B = b->num_seqs, R = b->num_logit_rows;
  if (T < 0 || B < 0 || R < 0) return fail(VD_ERR_INVALID_ARG, "negative size");
  if (T > t->max_tokens || B > c.max_seqs || R > c.max_logit_rows)
    return fail(VD_ERR_CAPACITY, "plan exceeds max_tokens, max_seqs or max_logit_rows");
  if (T == 0 && B == 0) {
    if (R > 0) return fail(VD_ERR_OUT_OF_RANGE, "logit row out of range");
    t->d = Desc{};
    t->planned = true;
    t->has_tokens = true;
    t->pool_id = pool->id;
    t->cache_id = cache->id;
    return VD_OK;
  }
  if (B == 0 || !b->cu_q || !b->cached_len || !b->open_table) return fail(VD_ERR_INVALID_ARG, "missing descriptor array");
  if (R > 0 && !b->logit_rows) return fail(VD_ERR_INVALID_ARG, "missing logit_rows");
  if (b->cu_q[0] != 0 || b->cu_q[B] != T) return fail(VD_ERR_INVALID_ARG, "cu_q must run from 0 to num_tokens");
  // lengths, table widths, page ids
  int stride = 0, open_stride = 0, splits = 1, n_seal = 0, most_q = 1, most_dec = 0;
  for (int i = 0; i < B; ++i) {
    const int ql = b->cu_q[i + 1] - b->cu_q[i], cached = b->cached_len[i];
    if (ql < 1 || b->cu_q[i + 1] > T) return fail(VD_ERR_INVALID_ARG, "every request needs q_len >= 1");
    if (cached < 0) return fail(VD_ERR_INVALID_ARG, "negative cached_len");
    const long long kv = static_cast<long long>(cached) + ql;
    if (kv > c.max_context) return fail(VD_ERR_CAPACITY, "request exceeds max_context");
    const int full = static_cast<int>(kv / 16), first = cached / 16, open = static_cast<int>((kv + 15) / 16) - first;
    if (full > 0 && !b->page_table) return fail(VD_ERR_INVALID_ARG, "missing page_table");
    if (full > b->page_table_stride || open > b->open_stride)
      return fail(VD_ERR_OUT_OF_RANGE, "page table narrower than the request");
    stride = std::max(stride, full);
    open_stride = std::max(open_stride, open);
    splits = std::max(splits, static_cast<int>((kv - 1) / kAttn8Split) + 1);
    n_seal += full - first;
    if (ql * m->G <= 16) {
      most_q = std::max(most_q, ql);
      most_dec = std::max(most_dec, ql * m->G);
    }
  }
  for (int k = 0; b->token_ids && k < T; ++k)
    if (b->token_ids[k] < 0 || b->token_ids[k] >= c.vocab) return fail(VD_ERR_OUT_OF_RANGE, "token id out of range");
  for (int j = 0; j < R; ++j)
    if (b->logit_rows[j] < 0 || b->logit_rows[j] >= T) return fail(VD_ERR_OUT_OF_RANGE, "logit row out of range");
  std::vector<unsigned char> sealed(cache->num_pages, 0);  // pages that the step seals
  std::unordered_set<long long> written;
  written.reserve(static_cast<size_t>(T) * 2);
  for (int i = 0; i < B; ++i) {
    const int ql = b->cu_q[i + 1] - b->cu_q[i], cached = b->cached_len[i], first = cached / 16;
    const int* ot = b->open_table + static_cast<size_t>(i) * b->open_stride;
    for (int j = 0; j < (cached + ql + 15) / 16 - first; ++j)
      if (ot[j] < 0 || ot[j] >= pool->num_pages) return fail(VD_ERR_OUT_OF_RANGE, "page id of the open table out of range");
    for (int k = 0; k < ql; ++k) {
      const int pos = cached + k;
      if (!written.insert(static_cast<long long>(ot[pos / 16 - first]) * 16 + (pos & 15)).second)
        return fail(VD_ERR_INVALID_ARG, "two new tokens of the step write the same KV slot");
    }
    for (int j = first; j < (cached + ql) / 16; ++j) {
      const int pg = b->page_table[static_cast<size_t>(i) * b->page_table_stride + j];
      if (pg < 0 || pg >= cache->num_pages) return fail(VD_ERR_OUT_OF_RANGE, "page id out of range");
      if (sealed[pg]) return fail(VD_ERR_INVALID_ARG, "a page of the cache is sealed twice");
      sealed[pg] = 1;
    }
  }
  for (int i = 0; i < B; ++i) {
    const int* pt = b->page_table + static_cast<size_t>(i) * b->page_table_stride;
    for (int j = 0; j < b->cached_len[i] / 16; ++j) {
      if (pt[j] < 0 || pt[j] >= cache->num_pages) return fail(VD_ERR_OUT_OF_RANGE, "page id out of range");
      if (sealed[pt[j]]) return fail(VD_ERR_INVALID_ARG, "the step seals a page that a row sees as an earlier one");
    }
  }

  // the image
  Desc d;
  d.T = T;
  d.B = B;
  d.R = R;
  d.stride = stride;
  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t o = off;
    off += n;
    return static_cast<int>(o);
  };
  // Attention blocks: 16 rows and a split on mma.sync for decode-shaped requests
  // and short chunks, 128 rows and a run of splits on tcgen05 for the rest; for
  // global layers and, without the splits that the window hides, for local ones.
  std::vector<int> blocks[6];
  const bool windowed = c.sliding_window > 0 && c.local_global_period > 0;
  std::vector<unsigned char> tc(B, 0);
  // Images of request i: of all its chunks, and again of those that hold own pages.
  auto images_of = [&](int i) {
    const int cached = b->cached_len[i], all = (cached + b->cu_q[i + 1] - b->cu_q[i] + 127) / 128;
    return 2 * all - cached / 128;
  };
  if (m->prefill_kernel == 0 && t->prefill != 1) {
    // What a chunk's (row block, KV head, 128 keys) units cost, in us at head dim 128:
    // 0.0095 for each of 16 rows on mma.sync; on tcgen05 0.02 for each of 128 rows and
    // as much for the keys' image, and 9 more for the launch.  (From a sweep of 48 shapes,
    // 1 to 32 requests of 5 to 1024 tokens behind 0 to 8000, 32 heads over 8.  mma.sync
    // against tcgen05, with today's kernels: 1 x 64 behind 1000 20 against 23 us; 1 x 512
    // behind 0 47 against 27; 32 x 8 behind 500 to 4000 106 against 192; 9 x 77 behind up
    // to 2500 157 against 70; 2 x 128 behind 3000 136 against 54; 8 heads over 4 of 256:
    // 1 x 512 behind 4000 204 against 94, 32 x 32 behind 100 to 1000 84 against 114.  The
    // rule takes the faster one but for near ties and, 32 heads over 8, 1 x 256 behind 0, 25
    // against 20.)  Where global and local layers take turns, one choice serves both, by
    // what the global ones cost.
    struct Choice {
      double more;    // what tcgen05 gains
      size_t images;  // bytes that it takes
      double rate;    // the former per byte
      int i;
    };
    std::vector<Choice> choices;
    for (int i = 0; i < B; ++i) {
      const int ql = b->cu_q[i + 1] - b->cu_q[i], rows = ql * m->G, all = (b->cached_len[i] + ql + 127) / 128;
      const int seen = windowed && c.local_global_period > c.n_layers ? std::min(all, (c.sliding_window + ql + 127) / 128) : all;
      const double unit = seen * c.n_kv_heads * (c.head_dim / 128.0);
      const double more = unit * (0.0095 * ((rows + 15) / 16) - 0.02 * ((rows + 127) / 128 + 1));
      if (rows > 16 && (more > 0 || t->prefill == 2)) {
        const size_t images = images_of(i) * static_cast<size_t>(c.n_kv_heads) * attn8_image_bytes(c.head_dim);
        choices.push_back({more, images, more / images, i});
      }
    }
    std::sort(choices.begin(), choices.end(),
              [](const Choice& x, const Choice& y) { return x.rate != y.rate ? x.rate > y.rate : x.i < y.i; });
    double gain = 0;
    size_t bytes = 0;
    for (const Choice& x : choices) {
      if (t->prefill == 0 && bytes + x.images > kMostImageBytes) continue;
      tc[x.i] = 1;
      gain += x.more;
      bytes += x.images;
    }
    if (gain < 9 && t->prefill == 0) std::fill(tc.begin(), tc.end(), 0);
  }
  // The tcgen05 blocks' requests have images of their chunks: of chunk 0 on, then of
  // those that hold own pages, numbered one request after the other.
  std::vector<int> image0(B, 0), chunks[2];
  long long n_images = 0;
  for (int i = 0; i < B; ++i) {
    const int ql = b->cu_q[i + 1] - b->cu_q[i], cached = b->cached_len[i], kv = cached + ql, all = (kv + 127) / 128;
    if (!tc[i]) continue;
    image0[i] = static_cast<int>(n_images);
    for (int local = 0; local <= (windowed ? 1 : 0); ++local) {
      const int first = local ? std::max(0, cached - c.sliding_window + 1) / 128 : 0;
      for (int ch = first; ch < all; ++ch) chunks[local].insert(chunks[local].end(), {i, ch, image0[i] + ch, 0, cached, kv, 0, 0});
      for (int ch = cached / 128; ch < all; ++ch)
        chunks[local].insert(chunks[local].end(), {i, ch, image0[i] + all + ch - cached / 128, 1, cached, kv, 0, 0});
    }
    n_images += images_of(i);
    if (n_images * c.n_kv_heads > 0x3fffffff) return fail(VD_ERR_CAPACITY, "plan too large");
  }
  // Of the tcgen05 row blocks, as many as fill the SMs in whole rounds take all of
  // their splits and need no merge; those of the last, partial round are cut into
  // runs of splits, so that it takes less of a round.  (A token's heads are in one
  // block, or the cut moves back to where they are.)

  std::vector<int> merge[2];  // tokens that the merge kernel folds
  for (int local = 0; local <= (windowed ? 1 : 0); ++local) {
    auto splits_of = [&](int i, int r0, int step, int* first) {
      const int cached = b->cached_len[i], rows = (b->cu_q[i + 1] - b->cu_q[i]) * m->G;
      *first = local ? std::max(0, cached + r0 / m->G - c.sliding_window + 1) / kAttn8Split : 0;
      return (cached + (std::min(rows, r0 + step) - 1) / m->G) / kAttn8Split + 1 - *first;
    };
    std::vector<std::pair<int, int>> rb;  // (request, first row) of the row blocks
    for (int i = 0; i < B; ++i) {
      const int q0 = b->cu_q[i], ql = b->cu_q[i + 1] - q0, cached = b->cached_len[i], rows = ql * m->G;
      if (tc[i]) {
        for (int r0 = 0; r0 < rows; r0 += 128) rb.emplace_back(i, r0);
        continue;
      }
      const int part0 = static_cast<int>(merge[local].size());
      for (int k = 0; k < ql; ++k) merge[local].push_back(q0 + k);
      std::vector<int>& to = blocks[3 * local + (rows > 16)];
      for (int r0 = 0; r0 < rows; r0 += 16) {
        int first;
        const int n = splits_of(i, r0, 16, &first);
        for (int k = 0; k < n; ++k) to.insert(to.end(), {i, q0, ql, cached, first + k, r0, 0, part0});
      }
    }
    const int n_rb = static_cast<int>(rb.size()), ctas = c.n_kv_heads * (c.head_dim > 128 ? 2 : 1);  // CTAs of a row block
    int direct = static_cast<int>(static_cast<long long>(n_rb) * ctas / m->n_sm * m->n_sm / ctas);
    while (direct < n_rb && direct > 0 && rb[direct].second % m->G) --direct;
    // runs that the others are cut into: as many as SMs
    const int parts_of = n_rb > direct ? std::max(1, m->n_sm / ((n_rb - direct) * ctas)) : 1;
    int part0 = 0;
    for (int j = 0; j < n_rb; ++j) {
      const int i = rb[j].first, r0 = rb[j].second, q0 = b->cu_q[i], ql = b->cu_q[i + 1] - q0, rows = ql * m->G;
      int first;
      const int n = splits_of(i, r0, 128, &first), parts = j < direct ? 1 : std::min(parts_of, n);
      // (a request's blocks that leave partials follow each other, and so do their tokens)
      if (j >= direct && (j == direct || rb[j - 1].first != i))
        part0 = static_cast<int>(merge[local].size()) - (r0 + m->G - 1) / m->G;
      for (int k = 0; k < parts; ++k)
        blocks[3 * local + 2].insert(blocks[3 * local + 2].end(),
                                     {image0[i], q0, ql, b->cached_len[i], first + n * k / parts, r0, first + n * (k + 1) / parts,
                                      j < direct ? kAttn8Folds : part0});
      if (j >= direct)  // the tokens whose first head is in the block
        for (int t0 = (r0 + m->G - 1) / m->G; t0 * m->G < std::min(rows, r0 + 128); ++t0) merge[local].push_back(q0 + t0);
    }
  }
  for (int k = 0; k < 6; ++k) {  // int4, then int2: first, for their alignment
    if (blocks[k].size() / 8 * c.n_kv_heads > 0x7fffffff) return fail(VD_ERR_CAPACITY, "plan too large");
    d.items[k] = take(blocks[k].size());
    d.n_items[k] = static_cast<int>(blocks[k].size() / 8);
  }
  for (int k = 0; k < 2; ++k) {
    d.chunks[k] = take(chunks[k].size());
    d.n_chunks[k] = static_cast<int>(chunks[k].size() / 8);
  }
  for (int k = 0; k < 2; ++k) d.split_pages[k] = take(kSplitPages * static_cast<size_t>(d.n_items[3 * k]));
  d.seal = take(2 * static_cast<size_t>(n_seal));
  d.n_seal = n_seal;
  d.tokens = take(T);
  d.positions = take(T);
  d.slot_page = take(T);
  d.logit_rows = take(R);
  for (int k = 0; k < 2; ++k) {
    d.merge_list[k] = take(merge[k].size());
    d.n_merge_kv8[k] = static_cast<int>(merge[k].size());
    d.merge_all[k] = d.n_merge_kv8[k] == T && std::is_sorted(merge[k].begin(), merge[k].end());
  }
  d.open_stride = open_stride;
  d.open_table = take(static_cast<size_t>(B) * open_stride);
  d.page_table = take(static_cast<size_t>(B) * stride);
  if (off > (1u << 30)) return fail(VD_ERR_CAPACITY, "plan too large");
  d.total = static_cast<int>(off);
  d.part_splits = splits;
  d.own_slots = most_q > 1 ? 2 : 1;
  d.lower8 = most_dec <= 8;
  const int slot = t->slot;
  VD_CUDA_TRY(cudaEventSynchronize(t->uploaded[slot]));  // this staging buffer's previous copy is done
  if (t->host_cap[slot] < off) {
    if (t->host[slot]) cudaFreeHost(t->host[slot]);
    t->host[slot] = nullptr;
    t->host_cap[slot] = 0;
    VD_CUDA_TRY(cudaMallocHost(reinterpret_cast<void**>(&t->host[slot]), off * 2 * sizeof(int)));
    t->host_cap[slot] = off * 2;
  }
  // Partials, of the tokens that the merge kernel folds (a long prompt's blocks fold
  // most of their own); global and local layers take turns in them.
  const size_t rows = std::max(merge[0].size(), merge[1].size()) * c.n_heads * splits;
  const size_t images = static_cast<size_t>(n_images) * c.n_kv_heads * attn8_image_bytes(c.head_dim);
  int rc;
  if (off > t->dev_cap || rows * (c.head_dim + 2) > t->part_cap || images > t->images_cap)
    t->planned = false;  // the old plan's buffers go
  if ((rc = grow(&t->dev, &t->dev_cap, off)) || (rc = grow(&t->part, &t->part_cap, rows * (c.head_dim + 2))) ||
      (rc = grow(&t->images, &t->images_cap, images)))
    return rc;
  int* h = t->host[slot];
  int ns = 0;
  for (int i = 0; i < B; ++i) {
    const int q0 = b->cu_q[i], ql = b->cu_q[i + 1] - q0, cached = b->cached_len[i], first = cached / 16;
    const int full = (cached + ql) / 16, open = (cached + ql + 15) / 16 - first;
    for (int j = 0; j < stride; ++j)
      h[d.page_table + static_cast<size_t>(i) * stride + j] =
          j < full ? b->page_table[static_cast<size_t>(i) * b->page_table_stride + j] : 0;
    for (int j = 0; j < open_stride; ++j)
      h[d.open_table + static_cast<size_t>(i) * open_stride + j] =
          j < open ? b->open_table[static_cast<size_t>(i) * b->open_stride + j] : 0;
    for (int j = first; j < full; ++j, ++ns) {
      h[d.seal + 2 * ns] = h[d.open_table + static_cast<size_t>(i) * open_stride + j - first];
      h[d.seal + 2 * ns + 1] = h[d.page_table + static_cast<size_t>(i) * stride + j];
    }
    for (int k = 0; k < ql; ++k) {
      h[d.tokens + q0 + k] = b->token_ids ? b->token_ids[q0 + k] : 0;
      h[d.positions + q0 + k] = cached + k;
      h[d.slot_page + q0 + k] = h[d.open_table + static_cast<size_t>(i) * open_stride + (cached + k) / 16 - first];
    }
  }
  for (int k = 0; k < 6; ++k) std::copy(blocks[k].begin(), blocks[k].end(), h + d.items[k]);
  for (int k = 0; k < 2; ++k)
    for (int n = 0; n < d.n_items[3 * k]; ++n) {
      const int* item = blocks[3 * k].data() + 8 * static_cast<size_t>(n);
      const int i = item[0], j0 = item[4] * kSplitPages;
      for (int j = 0; j < kSplitPages; ++j)  // (a row of the image's table is zero behind the request's pages)
        h[d.split_pages[k] + static_cast<size_t>(n) * kSplitPages + j] =
            j0 + j < stride ? h[d.page_table + static_cast<size_t>(i) * stride + j0 + j] : 0;
    }
  for (int k = 0; k < 2; ++k) std::copy(chunks[k].begin(), chunks[k].end(), h + d.chunks[k]);
  for (int j = 0; j < R; ++j) h[d.logit_rows + j] = b->logit_rows[j];
  for (int k = 0; k < 2; ++k) std::copy(merge[k].begin(), merge[k].end(), h + d.merge_list[k]);
  d.images = t->images;
  d.base = t->dev;
  d.part_o = t->part;
  d.part_ml = t->part + rows * c.head_dim;
  d.kv8 = cache;
  t->planned = false;  // until the new plan is on its way
  VD_CUDA_TRY(cudaMemcpyAsync(t->dev, h, off * sizeof(int), cudaMemcpyHostToDevice, s));
  VD_CUDA_TRY(cudaEventRecord(t->uploaded[slot], s));
  t->slot ^= 1;
  t->d = d;
  t->pool_id = pool->id;
  t->cache_id = cache->id;
  t->has_tokens = b->token_ids != nullptr;
  t->planned = true;
  return VD_OK;
}

}  // namespace

int vd::run_kv8_seal(vd_model* m, vd_kv_pool* pool, int layer, const Desc& d, cudaStream_t s) {
  if (d.n_seal == 0) return VD_OK;
  Prof p(m, K_ROPE, s);
  PagePairs pairs;
  pairs.dev = reinterpret_cast<const int2*>(d.base + d.seal);
  pairs.n = d.n_seal;
  return launch_kv8_seal(seal_args(d.kv8, pool, layer), pairs, false, s);
}

int vd::run_kv8_attention(vd_model* m, vd_kv_pool* pool, int layer, const Desc& d, const __nv_bfloat16* q,
                          __nv_bfloat16* out, cudaStream_t s) {
  const vd_model_config& c = m->cfg;
  Attn8Args a{};
  a.q = q;
  a.part_o = d.part_o;
  a.part_ml = d.part_ml;
  a.page_table = d.base + d.page_table;
  a.open_table = d.base + d.open_table;
  a.codes = d.kv8->codes(layer);
  a.scales = d.kv8->scales(layer);
  a.pt_stride = d.stride;
  a.open_stride = d.open_stride;
  a.Hq = c.n_heads;
  a.Hkv = c.n_kv_heads;
  a.images = d.images;
  a.out = out;
  a.open = static_cast<const __nv_bfloat16*>(pool->data) +
           static_cast<size_t>(layer) * pool->num_pages * 2 * c.n_kv_heads * 16 * c.head_dim;
  a.layer_row0 = static_cast<int>(static_cast<long long>(layer) * pool->num_pages * 2 * c.n_kv_heads * 16);
  a.window = layer_is_local(c, layer) ? c.sliding_window : 0;
  a.chunks = reinterpret_cast<const int4*>(d.base + d.chunks[a.window > 0]);
  a.max_splits = d.part_splits;
  a.scale_log2 = static_cast<float>(1.4426950408889634 / sqrt(static_cast<double>(c.head_dim)));
  a.status = m->status;
  int rc;
  const int local = a.window > 0;
  for (int cls = 0; cls < 3; ++cls) {
    const int k = 3 * local + cls;
    if (d.n_items[k] == 0) continue;
    Prof p(m, K_ATTN, s);
    p.kernels = cls == 2 ? 2 : 1;
    a.items = reinterpret_cast<const int4*>(d.base + d.items[k]);
    a.own_slots = cls ? 2 : d.own_slots;
    a.split_pages = cls ? nullptr : d.base + d.split_pages[local];
    if ((rc = cls == 2 ? launch_attention8_tc(a, c.head_dim, d.kv8->format, d.n_chunks[local], d.n_items[k], s)
                       : launch_attention8(pool->map, a, c.head_dim, d.kv8->format, !cls && d.lower8, d.n_items[k], s)))
      return rc;
  }
  const int n_merge = d.n_merge_kv8[local];
  if (n_merge == 0) return VD_OK;  // every row's splits were folded by its block
  MergeArgs g{};
  g.tokens = d.merge_all[local] ? nullptr : d.base + d.merge_list[local];
  g.by_rank = true;
  g.part_o = d.part_o;
  g.part_ml = d.part_ml;
  g.out = out;
  g.positions = d.base + d.positions;
  g.T = n_merge;
  g.Hq = c.n_heads;
  g.window = a.window;
  g.split = kAttn8Split;
  g.max_splits = d.part_splits;
  Prof p(m, K_MERGE, s);
  return launch_merge(g, c.head_dim, s);
}

extern "C" {

size_t vd_kv8_bytes(const vd_model* m, int32_t num_pages) {
  if (!m || num_pages < 0) return 0;
  return static_cast<size_t>(m->cfg.n_layers) * num_pages * m->cfg.n_kv_heads * (32 * m->cfg.head_dim + 16);
}

int vd_kv8_create(vd_model* m, int32_t format, int32_t num_pages, void* dev_mem, size_t bytes, vd_kv8** out) {
  if (!out) return fail(VD_ERR_INVALID_ARG, "null argument");
  *out = nullptr;
  if (check_model(m)) return VD_ERR_INVALID_ARG;
  if (format != VD_KV8_INT8 && format != VD_KV8_E4M3) return fail(VD_ERR_INVALID_ARG, "format: VD_KV8_INT8 or VD_KV8_E4M3");
  if (num_pages < 1) return fail(VD_ERR_INVALID_ARG, "num_pages must be >= 1");
  if (const int rc = check_device(m)) return rc;
  const size_t need = vd_kv8_bytes(m, num_pages);
  if (dev_mem && bytes < need) return fail(VD_ERR_CAPACITY, "dev_mem smaller than vd_kv8_bytes()");
  if (reinterpret_cast<uintptr_t>(dev_mem) & 255) return fail(VD_ERR_INVALID_ARG, "dev_mem must be 256-byte aligned");
  if (dev_mem) {
    cudaPointerAttributes at{};
    VD_CUDA_TRY(cudaPointerGetAttributes(&at, dev_mem));
    if (!(at.type == cudaMemoryTypeManaged || (at.type == cudaMemoryTypeDevice && at.device == m->device)))
      return fail(VD_ERR_INVALID_ARG, "dev_mem is not memory of the model's device");
  }
  vd_kv8* c = new (std::nothrow) vd_kv8();
  if (!c) return fail(VD_ERR_CAPACITY, "out of host memory");
  static std::atomic<unsigned long long> next_id{1};
  c->m = m;
  c->id = next_id++;
  c->device = m->device;
  c->format = format;
  c->num_pages = num_pages;
  c->data = dev_mem;
  if (!dev_mem) {
    if (cudaMalloc(&c->data, need) != cudaSuccess) {
      delete c;
      return fail(VD_ERR_CUDA, "cudaMalloc(8-bit cache) failed");
    }
    c->owned = true;
  }
  if (cudaMemset(c->data, 0, need) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
    vd_destroy_kv8(c);
    return fail(VD_ERR_CUDA, "cudaMemset(8-bit cache) failed");
  }
  *out = c;
  return VD_OK;
}

void vd_destroy_kv8(vd_kv8* c) {
  if (!c) return;
  if (c->owned && c->data) {
    int dev = c->device;
    cudaGetDevice(&dev);
    if (dev != c->device) cudaSetDevice(c->device);
    cudaDeviceSynchronize();
    cudaFree(c->data);
    if (dev != c->device) cudaSetDevice(dev);
  }
  delete c;
}

void* vd_kv8_data(vd_kv8* c) { return c ? c->data : nullptr; }

int vd_kv8_seal(vd_kv8* c, vd_kv_pool* pool, int32_t layer, int32_t n, const int32_t* src, const int32_t* dst,
                void* stream) {
  return guarded([&] { return seal_call(c, pool, layer, n, src, dst, false, stream); });
}
int vd_kv8_unseal(vd_kv8* c, vd_kv_pool* pool, int32_t layer, int32_t n, const int32_t* src, const int32_t* dst,
                  void* stream) {
  return guarded([&] { return seal_call(c, pool, layer, n, src, dst, true, stream); });
}

int vd_kv8_plan_create(vd_model* m, int32_t max_tokens, vd_kv8_plan** out) {
  if (!out) return fail(VD_ERR_INVALID_ARG, "null argument");
  *out = nullptr;
  if (check_model(m)) return VD_ERR_INVALID_ARG;
  if (max_tokens < 1) return fail(VD_ERR_INVALID_ARG, "max_tokens must be >= 1");
  if (max_tokens > m->cfg.max_tokens) return fail(VD_ERR_CAPACITY, "max_tokens exceeds the model's");
  if (const int rc = check_device(m)) return rc;
  vd_kv8_plan* t = new (std::nothrow) vd_kv8_plan();
  if (!t) return fail(VD_ERR_CAPACITY, "out of host memory");
  t->m = m;
  t->device = m->device;
  t->max_tokens = max_tokens;
  for (cudaEvent_t& e : t->uploaded)
    if (cudaEventCreateWithFlags(&e, cudaEventDisableTiming) != cudaSuccess) {
      vd_destroy_kv8_plan(t);
      return fail(VD_ERR_CUDA, "cudaEventCreate failed");
    }
  *out = t;
  return VD_OK;
}

void vd_destroy_kv8_plan(vd_kv8_plan* t) {
  if (!t) return;
  int dev = t->device;  // the caller's current device, put back below
  cudaGetDevice(&dev);
  if (dev != t->device) cudaSetDevice(t->device);
  cudaDeviceSynchronize();
  for (int k = 0; k < 2; ++k) {
    if (t->host[k]) cudaFreeHost(t->host[k]);
    if (t->uploaded[k]) cudaEventDestroy(t->uploaded[k]);
  }
  if (t->dev) cudaFree(t->dev);
  if (t->part) cudaFree(t->part);
  if (t->images) cudaFree(t->images);
  if (dev != t->device) cudaSetDevice(dev);
  delete t;
}

int vd_kv8_plan_make(vd_kv8_plan* p, vd_kv8* c, vd_kv_pool* pool, const vd_kv8_batch* b, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (const int rc = check_call(p, c, pool, s)) return rc;
  return guarded([&] { return make_plan(p, c, pool, b, s); });
}

int vd_kv8_set_prefill(vd_kv8_plan* p, int32_t kernel) {
  if (!p) return fail(VD_ERR_INVALID_ARG, "null plan");
  if (kernel < 0 || kernel > 2) return fail(VD_ERR_INVALID_ARG, "kernel must be 0, 1 or 2");
  p->prefill = kernel;
  return VD_OK;
}

int vd_op_kv8_rope_kv(vd_kv8_plan* p, vd_kv8* c, vd_kv_pool* pool, int32_t layer, const void* qkv, void* q_out,
                      void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int rc;
  if ((rc = check_planned(p, c, pool, s)) || (rc = check_layer(p->m, layer))) return rc;
  if (p->d.T == 0) return VD_OK;
  if (!qkv || !q_out) return fail(VD_ERR_INVALID_ARG, "null argument");
  if (!aligned16(qkv) || !aligned16(q_out)) return fail(VD_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
  return run_rope(p->m, pool, layer, p->d, static_cast<const __nv_bfloat16*>(qkv), static_cast<__nv_bfloat16*>(q_out), s);
}

int vd_op_kv8_seal(vd_kv8_plan* p, vd_kv8* c, vd_kv_pool* pool, int32_t layer, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int rc;
  if ((rc = check_planned(p, c, pool, s)) || (rc = check_layer(p->m, layer))) return rc;
  return p->d.T == 0 ? VD_OK : run_kv8_seal(p->m, pool, layer, p->d, s);
}

int vd_op_kv8_attention(vd_kv8_plan* p, vd_kv8* c, vd_kv_pool* pool, int32_t layer, const void* q, void* out,
                        void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int rc;
  if ((rc = check_planned(p, c, pool, s)) || (rc = check_layer(p->m, layer))) return rc;
  if (p->d.T == 0) return VD_OK;
  if (!q || !out) return fail(VD_ERR_INVALID_ARG, "null argument");
  if (!aligned16(q) || !aligned16(out)) return fail(VD_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
  const uintptr_t qa = reinterpret_cast<uintptr_t>(q), oa = reinterpret_cast<uintptr_t>(out);
  const size_t bytes = static_cast<size_t>(p->d.T) * p->m->cfg.n_heads * p->m->cfg.head_dim * 2;
  if (qa < oa + bytes && oa < qa + bytes)  // (blocks that write their rows' outputs run beside blocks that read queries)
    return fail(VD_ERR_INVALID_ARG, "q and out overlap");
  return run_kv8_attention(p->m, pool, layer, p->d, static_cast<const __nv_bfloat16*>(q),
                           static_cast<__nv_bfloat16*>(out), s);
}

int vd_step_kv8(vd_kv8_plan* p, vd_kv8* c, vd_kv_pool* pool, float* logits_out, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (const int rc = check_planned(p, c, pool, s)) return rc;
  if (!p->has_tokens) return fail(VD_ERR_INVALID_ARG, "the plan has no token_ids");
  if (p->d.T == 0) return VD_OK;
  if (p->d.R > 0 && (!logits_out || !aligned16(logits_out)))
    return fail(VD_ERR_INVALID_ARG, "logits_out null or not 16-byte aligned");
  return enqueue_step(p->m, pool, p->d, logits_out, nullptr, s);
}

int vd_kv_copy_pages(vd_kv_pool* pool, int32_t n, const int32_t* src, const int32_t* dst, void* stream) {
  if (!pool) return fail(VD_ERR_INVALID_ARG, "null pool");
  return guarded([&]() -> int {
    int rc;
    if ((rc = check_device(pool->m)) || (rc = check_pages(n, src, dst, pool->num_pages, pool->num_pages, true))) return rc;
    const vd_model_config& f = pool->m->cfg;
    CopyArgs a{};
    a.data = static_cast<uint8_t*>(pool->data);
    a.bytes = 2LL * f.n_kv_heads * 16 * f.head_dim * 2;
    a.layer = a.bytes * pool->num_pages;
    a.layers = f.n_layers;
    return for_pairs(n, src, dst, [&](const auto& p) { return launch_copy_pages(a, p, static_cast<cudaStream_t>(stream)); });
  });
}

int vd_kv8_copy_pages(vd_kv8* c, int32_t n, const int32_t* src, const int32_t* dst, void* stream) {
  if (!c) return fail(VD_ERR_INVALID_ARG, "null cache");
  return guarded([&]() -> int {
    int rc;
    if ((rc = check_device(c->m)) || (rc = check_pages(n, src, dst, c->num_pages, c->num_pages, true))) return rc;
    const vd_model_config& f = c->m->cfg;
    CopyArgs a{};
    a.data = c->codes(0);
    a.bytes = 32LL * f.n_kv_heads * f.head_dim;
    a.layer = c->codes_layer();
    a.extra = c->scales(0);
    a.extra_layer = c->scales_layer();
    a.n_extra = f.n_kv_heads;
    a.layers = f.n_layers;
    return for_pairs(n, src, dst, [&](const auto& p) { return launch_copy_pages(a, p, static_cast<cudaStream_t>(stream)); });
  });
}

}  // extern "C"
