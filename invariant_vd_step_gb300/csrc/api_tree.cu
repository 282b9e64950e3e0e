// C ABI of the token trees (vd_tree): planning, attention, RoPE + K/V write,
// a whole step over the nodes, and acceptance.
#include <math.h>

#include <algorithm>
#include <string>
#include <unordered_set>
#include <vector>

#include "vd_device.cuh"
#include "vd_internal.h"
#include "vd_model.h"

using namespace vd;

struct vd_tree {
  vd_model* m = nullptr;
  int device = 0;  // the model's
  int max_nodes = 0;
  // the plan in force
  Desc d;
  unsigned long long pool_id = 0;
  bool planned = false, has_tokens = false;
  // device copy of the plan and split partials; both grow with the plans
  int* dev = nullptr;
  size_t dev_cap = 0;  // ints
  float* part = nullptr;
  size_t part_cap = 0;  // floats
  int* host[2] = {nullptr, nullptr};  // pinned staging
  size_t host_cap[2] = {0, 0};
  cudaEvent_t uploaded[2] = {nullptr, nullptr};
  int slot = 0;
};

namespace {

// Rows (nodes x query heads per KV head) of a CTA of each class, the same
// bits in every one.
constexpr int kClsRows[4] = {16, 32, 64, 128};

int check_call(const vd_tree* t, const vd_kv_pool* pool, cudaStream_t s) {
  if (!t || !pool) return fail(VD_ERR_INVALID_ARG, "null tree or pool");
  if (pool->m != t->m) return fail(VD_ERR_INVALID_ARG, "the pool belongs to another model");
  int dev = -1;
  VD_CUDA_TRY(cudaGetDevice(&dev));
  if (dev != t->m->device) return fail(VD_ERR_INVALID_ARG, "the model lives on another device than the current one");
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  VD_CUDA_TRY(cudaStreamIsCapturing(s, &cap));
  if (cap != cudaStreamCaptureStatusNone)
    return fail(VD_ERR_UNSUPPORTED, "token-tree calls cannot be captured: their plan changes from step to step");
  return VD_OK;
}

int check_planned(const vd_tree* t, const vd_kv_pool* pool, cudaStream_t s) {
  if (const int rc = check_call(t, pool, s)) return rc;
  if (!t->planned) return fail(VD_ERR_INVALID_ARG, "the tree has no plan");
  if (t->pool_id != pool->id) return fail(VD_ERR_INVALID_ARG, "the tree was planned for another pool");
  return VD_OK;
}

// Grows a device buffer to at least n elements (the old one is freed once the
// device is done with it).
template <typename T>
int grow(T** p, size_t* cap, size_t n) {
  if (n <= *cap) return VD_OK;
  const size_t want = std::max(n, *cap + *cap / 2);
  if (*p) cudaFree(*p);
  *p = nullptr;
  *cap = 0;
  VD_CUDA_TRY(cudaMalloc(reinterpret_cast<void**>(p), want * sizeof(T)));
  *cap = want;
  return VD_OK;
}

}  // namespace

// The shared tiles of every request (three classes of CTA, by the request's
// rows), then each node's own tiles, then the fold of the splits.
int vd::run_tree_attention(vd_model* m, vd_kv_pool* pool, int layer, const Desc& d, const __nv_bfloat16* q,
                           __nv_bfloat16* out, cudaStream_t s) {
  const vd_model_config& c = m->cfg;
  const int hd = c.head_dim;
  AttnArgs a{};
  a.q = q;
  a.part_o = d.part_o;
  a.part_ml = d.part_ml;
  a.cu_q = d.base + d.cu_q;
  a.cached_len = d.base + d.cached;
  a.page_table = d.base + d.page_table;
  a.pt_stride = d.stride;
  a.Hq = c.n_heads;
  a.Hkv = c.n_kv_heads;
  a.layer_row0 = static_cast<int>(static_cast<long long>(layer) * pool->num_pages * 2 * c.n_kv_heads * 16);
  a.pool_rows = static_cast<int>(pool->rows);
  a.window = layer_is_local(c, layer) ? c.sliding_window : 0;
  a.split = m->split;
  a.max_splits = d.part_splits;
  a.scale_log2 = static_cast<float>(1.4426950408889634 / sqrt(static_cast<double>(hd)));
  a.status = m->status;
  a.tree_pos = d.base + d.positions;
  int rc;
  Prof p(m, K_ATTN, s);
  p.kernels = 2;
  for (int k = 0; k < 4; ++k) {
    if (d.cls[k].items == 0) continue;
    ++p.kernels;
    a.cls_seq = d.base + d.cls[k].seq;
    a.cls_start = d.base + d.cls[k].start;
    a.n_cls = d.cls[k].n;
    if ((rc = k == 3 ? launch_attention_tc(pool->map_tc, a, hd, d.cls[k].items, s)
                     : launch_attention_tree(pool->map, a, hd, kClsRows[k], d.cls[k].items, s)))
      return rc;
  }
  TreeTailArgs t{};
  t.q = q;
  t.pool = static_cast<const __nv_bfloat16*>(pool->data) +
           static_cast<size_t>(layer) * pool->num_pages * 2 * c.n_kv_heads * 16 * hd;
  t.part_o = d.part_o;
  t.part_ml = d.part_ml;
  t.node_seq = d.base + d.node_seq;
  t.cu_q = a.cu_q;
  t.cached_len = a.cached_len;
  t.page_table = a.page_table;
  t.positions = a.tree_pos;
  t.path_off = d.base + d.path_off;
  t.path = d.base + d.path;
  t.T = d.T;
  t.Hq = a.Hq;
  t.Hkv = a.Hkv;
  t.pt_stride = d.stride;
  t.window = a.window;
  t.split = a.split;
  t.max_splits = a.max_splits;
  t.scale_log2 = a.scale_log2;
  t.status = m->status;
  t.blk_seq = d.base + d.blk_seq;
  t.blk_first = d.base + d.blk_first;
  t.n_blk = d.n_blk;
  t.npg = d.npg;
  t.tail_rows = d.tail_rows;
  // (with a window a CTA of the attention kernel may see no key and leave before its wait)
  t.early = a.window == 0 && d.cls[0].items + d.cls[1].items + d.cls[2].items + d.cls[3].items > 0;
  if ((rc = launch_tree_tail(t, hd, s))) return rc;
  MergeArgs g{};
  g.part_o = d.part_o;
  g.part_ml = d.part_ml;
  g.out = out;
  g.positions = a.tree_pos;
  g.T = d.T;
  g.Hq = c.n_heads;
  g.window = a.window;
  g.split = m->split;
  g.max_splits = d.part_splits;
  return launch_merge(g, hd, s);
}

extern "C" {

int vd_tree_create(vd_model* m, int32_t max_nodes, vd_tree** out) {
  if (check_model(m) || !out) return fail(VD_ERR_INVALID_ARG, "null argument");
  *out = nullptr;
  if (max_nodes < 1) return fail(VD_ERR_INVALID_ARG, "max_nodes must be >= 1");
  if (max_nodes > m->cfg.max_tokens) return fail(VD_ERR_CAPACITY, "max_nodes exceeds the model's max_tokens");
  int dev = -1;
  VD_CUDA_TRY(cudaGetDevice(&dev));
  if (dev != m->device) return fail(VD_ERR_INVALID_ARG, "the model lives on another device than the current one");
  vd_tree* t = new vd_tree();
  t->m = m;
  t->device = dev;
  t->max_nodes = max_nodes;
  for (cudaEvent_t& e : t->uploaded)
    if (cudaEventCreateWithFlags(&e, cudaEventDisableTiming) != cudaSuccess) {
      vd_destroy_tree(t);
      return fail(VD_ERR_CUDA, "cudaEventCreate failed");
    }
  *out = t;
  return VD_OK;
}

void vd_destroy_tree(vd_tree* t) {
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
  if (dev != t->device) cudaSetDevice(dev);
  delete t;
}

int vd_tree_plan(vd_tree* t, vd_kv_pool* pool, const vd_tree_batch* b, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (const int rc = check_call(t, pool, s)) return rc;
  vd_model* m = t->m;
  const vd_model_config& c = m->cfg;
  if (!b) return fail(VD_ERR_INVALID_ARG, "null batch");
  const int T = b->num_nodes, B = b->num_seqs;
  if (T < 0 || B < 0) return fail(VD_ERR_INVALID_ARG, "negative size");
  if (T > t->max_nodes || B > c.max_seqs) return fail(VD_ERR_CAPACITY, "plan exceeds max_nodes or max_seqs");
  if (T == 0 && B == 0) {
    t->d = Desc{};
    t->d.tree = true;
    t->planned = true;
    t->has_tokens = true;
    t->pool_id = pool->id;
    return VD_OK;
  }
  if (B == 0 || !b->cu_nodes || !b->parent || !b->cached_len || !b->page_table)
    return fail(VD_ERR_INVALID_ARG, "missing descriptor array");
  if (b->cu_nodes[0] != 0 || b->cu_nodes[B] != T) return fail(VD_ERR_INVALID_ARG, "cu_nodes must run from 0 to num_nodes");
  int stride = 0, splits = 1;
  size_t paths = 0;
  std::vector<int> depth(T);
  for (int i = 0; i < B; ++i) {
    const int n0 = b->cu_nodes[i], n1 = b->cu_nodes[i + 1];
    if (n1 <= n0 || n1 > T) return fail(VD_ERR_INVALID_ARG, "every request needs at least one node");
    if (n1 - n0 > kTreeMaxNodes) return fail(VD_ERR_CAPACITY, "a request's tree holds at most 1024 nodes");
    const int cached = b->cached_len[i];
    if (cached < 0) return fail(VD_ERR_INVALID_ARG, "negative cached_len");
    const long long kv = static_cast<long long>(cached) + (n1 - n0);
    if (kv > c.max_context) return fail(VD_ERR_CAPACITY, "request exceeds max_context");
    const int np = static_cast<int>((kv + 15) / 16);
    if (np > b->page_table_stride) return fail(VD_ERR_OUT_OF_RANGE, "page table narrower than the request");
    stride = std::max(stride, np);
    for (int k = n0; k < n1; ++k) {
      const int p = b->parent[k];
      if (k == n0 ? p != -1 : (p < 0 || p >= k - n0))
        return fail(VD_ERR_INVALID_ARG, "parent: -1 for a request's first node, else an earlier node of the request");
      depth[k] = k == n0 ? 0 : depth[n0 + p] + 1;
      paths += depth[k] + 1;
      splits = std::max(splits, (cached + depth[k]) / m->split + 1);
      if (b->token_ids && (b->token_ids[k] < 0 || b->token_ids[k] >= c.vocab))
        return fail(VD_ERR_OUT_OF_RANGE, "token id out of range");
    }
    for (int j = 0; j < np; ++j) {
      const int pg = b->page_table[static_cast<size_t>(i) * b->page_table_stride + j];
      if (pg < 0 || pg >= pool->num_pages) return fail(VD_ERR_OUT_OF_RANGE, "page id out of range");
    }
  }
  if (paths > (1u << 28)) return fail(VD_ERR_CAPACITY, "the trees' paths hold more than 2^28 nodes");
  std::unordered_set<long long> written;
  written.reserve(static_cast<size_t>(T) * 2);
  for (int i = 0; i < B; ++i)
    for (int k = b->cu_nodes[i]; k < b->cu_nodes[i + 1]; ++k) {
      const int slot = b->cached_len[i] + k - b->cu_nodes[i];
      const long long pg = b->page_table[static_cast<size_t>(i) * b->page_table_stride + slot / 16];
      if (!written.insert(pg * 16 + (slot & 15)).second)
        return fail(VD_ERR_INVALID_ARG, "two nodes of the plan have the same KV slot");
    }

  // the image: per-node arrays, per-request arrays, work classes, paths
  Desc d;
  d.tree = true;
  d.T = T;
  d.B = B;
  d.R = T;  // a step returns logits for every node
  d.stride = stride;
  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t o = off;
    off += n;
    return static_cast<int>(o);
  };
  d.tokens = take(T);
  d.positions = take(T);
  d.slot_page = take(T);
  d.slots = take(T);
  d.logit_rows = take(T);
  d.node_seq = take(T);
  d.path_off = take(T);
  d.parent = take(T);
  d.cu_q = take(B + 1);
  d.cached = take(B);
  for (auto& k : d.cls) {
    k.seq = take(B);
    k.start = take(B + 1);
  }
  for (int i = 0; i < B; ++i)
    d.tail_rows = std::max(d.tail_rows, b->cached_len[i] % m->key_tile + b->cu_nodes[i + 1] - b->cu_nodes[i]);
  int per_blk = 1;
  d.npg = tree_nodes_per_warp(c.head_dim, T, c.n_kv_heads, m->G, d.tail_rows, m->n_sm, &per_blk);
  for (int i = 0; i < B; ++i) d.n_blk += (b->cu_nodes[i + 1] - b->cu_nodes[i] + per_blk - 1) / per_blk;
  d.blk_seq = take(d.n_blk);
  d.blk_first = take(d.n_blk);
  d.path = take(paths);
  d.page_table = take(static_cast<size_t>(B) * stride);
  if (off > (1u << 30)) return fail(VD_ERR_CAPACITY, "plan too large");
  d.total = static_cast<int>(off);
  d.part_splits = splits;

  const int slot = t->slot;
  VD_CUDA_TRY(cudaEventSynchronize(t->uploaded[slot]));  // this staging buffer's previous copy is done
  if (t->host_cap[slot] < off) {
    if (t->host[slot]) cudaFreeHost(t->host[slot]);
    t->host[slot] = nullptr;
    t->host_cap[slot] = 0;
    VD_CUDA_TRY(cudaMallocHost(reinterpret_cast<void**>(&t->host[slot]), off * 2 * sizeof(int)));
    t->host_cap[slot] = off * 2;
  }
  const size_t rows = static_cast<size_t>(T) * c.n_heads * splits;
  int rc;
  t->planned = false;  // until the new plan is on its way
  if ((rc = grow(&t->dev, &t->dev_cap, off)) || (rc = grow(&t->part, &t->part_cap, rows * (c.head_dim + 2)))) return rc;
  int* h = t->host[slot];
  int npath = 0, nblk = 0;
  auto items = [&](int nodes, int shared, int rows_per_cta) {
    const int r = nodes * m->G, nsplit = shared > 0 ? (shared - 1) / m->split + 1 : 0;
    return (r + rows_per_cta - 1) / rows_per_cta * c.n_kv_heads * nsplit;
  };
  // A launch of at most one 16-row CTA per SM is bound by its CTAs' latency, not
  // by what they read: blocks of 16 rows (their K/V tiles shared by four warps)
  // then beat fewer CTAs of more rows (one tree of 8 nodes x 4 rows: 18 us, in
  // one block of 32 rows 26.7 us).  Larger launches take tcgen05 CTAs above 16
  // rows: 16 trees of 16 nodes x 4 rows 107 us, on mma.sync blocks of 64 127 us.
  long long small_items = 0;
  for (int i = 0; i < B; ++i)
    small_items += items(b->cu_nodes[i + 1] - b->cu_nodes[i], b->cached_len[i] / m->key_tile * m->key_tile, 16);
  for (int i = 0; i < B; ++i) {
    const int n0 = b->cu_nodes[i], n = b->cu_nodes[i + 1] - n0, cached = b->cached_len[i];
    for (int j = 0; j < stride; ++j)
      h[d.page_table + i * stride + j] =
          j < (cached + n + 15) / 16 ? b->page_table[static_cast<size_t>(i) * b->page_table_stride + j] : 0;
    for (int k = 0; k < n; ++k) {
      const int node = n0 + k, sl = cached + k;
      h[d.tokens + node] = b->token_ids ? b->token_ids[node] : 0;
      h[d.positions + node] = cached + depth[node];
      h[d.slot_page + node] = h[d.page_table + i * stride + sl / 16];
      h[d.slots + node] = sl & 15;
      h[d.logit_rows + node] = node;
      h[d.node_seq + node] = i;
      h[d.parent + node] = b->parent[node];
      h[d.path_off + node] = npath;
      if (depth[node] > 0) {  // the parent's path, then the node
        const int from = h[d.path_off + n0 + b->parent[node]];
        std::copy(h + d.path + from, h + d.path + from + depth[node], h + d.path + npath);
      }
      h[d.path + npath + depth[node]] = k;
      npath += depth[node] + 1;
    }
    h[d.cu_q + i] = n0;
    h[d.cached + i] = cached;
    for (int k = 0; k < n; k += per_blk, ++nblk) {
      h[d.blk_seq + nblk] = i;
      h[d.blk_first + nblk] = k;
    }
    // the request's class, by its rows
    const int shared = cached / m->key_tile * m->key_tile, r = n * m->G;
    const bool tc = m->prefill_kernel == 0 && attn_tc_supported(c.head_dim);
    const int k = r <= 16 || small_items <= m->n_sm ? 0 : tc ? 3 : r <= 32 ? 1 : 2;
    h[d.cls[k].seq + d.cls[k].n] = i;
    h[d.cls[k].start + d.cls[k].n] = d.cls[k].items;
    d.cls[k].items += items(n, shared, kClsRows[k]);
    ++d.cls[k].n;
  }
  h[d.cu_q + B] = T;
  for (const auto& k : d.cls) h[k.start + k.n] = k.items;
  d.base = t->dev;
  d.part_o = t->part;
  d.part_ml = t->part + rows * c.head_dim;
  VD_CUDA_TRY(cudaMemcpyAsync(t->dev, h, off * sizeof(int), cudaMemcpyHostToDevice, s));
  VD_CUDA_TRY(cudaEventRecord(t->uploaded[slot], s));
  t->slot ^= 1;
  t->d = d;
  t->pool_id = pool->id;
  t->has_tokens = b->token_ids != nullptr;
  t->planned = true;
  return VD_OK;
}

int vd_op_tree_attention(vd_tree* t, vd_kv_pool* pool, int32_t layer, const void* q, void* out, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (const int rc = check_planned(t, pool, s)) return rc;
  if (layer < 0 || layer >= t->m->cfg.n_layers) return fail(VD_ERR_OUT_OF_RANGE, "layer out of range");
  if (t->d.T == 0) return VD_OK;
  if (!q || !out) return fail(VD_ERR_INVALID_ARG, "null argument");
  if (!aligned16(q) || !aligned16(out)) return fail(VD_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
  return run_tree_attention(t->m, pool, layer, t->d, static_cast<const __nv_bfloat16*>(q),
                            static_cast<__nv_bfloat16*>(out), s);
}

int vd_op_tree_rope_kv(vd_tree* t, vd_kv_pool* pool, int32_t layer, const void* qkv, void* q_out, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (const int rc = check_planned(t, pool, s)) return rc;
  if (layer < 0 || layer >= t->m->cfg.n_layers) return fail(VD_ERR_OUT_OF_RANGE, "layer out of range");
  if (t->d.T == 0) return VD_OK;
  if (!qkv || !q_out) return fail(VD_ERR_INVALID_ARG, "null argument");
  if (!aligned16(qkv) || !aligned16(q_out)) return fail(VD_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
  return run_rope(t->m, pool, layer, t->d, static_cast<const __nv_bfloat16*>(qkv), static_cast<__nv_bfloat16*>(q_out),
                  s);
}

int vd_step_tree(vd_tree* t, vd_kv_pool* pool, float* logits_out, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (const int rc = check_planned(t, pool, s)) return rc;
  if (!t->has_tokens) return fail(VD_ERR_INVALID_ARG, "the plan has no token_ids");
  if (t->d.T == 0) return VD_OK;
  if (t->d.T > t->m->cfg.max_logit_rows) return fail(VD_ERR_CAPACITY, "the plan's nodes exceed max_logit_rows");
  if (!logits_out || !aligned16(logits_out)) return fail(VD_ERR_INVALID_ARG, "logits_out null or not 16-byte aligned");
  return enqueue_step(t->m, pool, t->d, logits_out, nullptr, s);
}

int vd_tree_accept(vd_tree* t, vd_kv_pool* pool, const int32_t* node_tokens, const int32_t* choices,
                   int32_t* accepted_len, int32_t* out_tokens, int32_t out_stride, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (const int rc = check_planned(t, pool, s)) return rc;
  if (t->d.T == 0) return VD_OK;
  if (!node_tokens && !t->has_tokens) return fail(VD_ERR_INVALID_ARG, "neither node_tokens nor token_ids in the plan");
  if (out_stride < 1) return fail(VD_ERR_CAPACITY, "out_stride must hold a path of at least one node");
  if (!choices || !accepted_len || !out_tokens) return fail(VD_ERR_INVALID_ARG, "null argument");
  if ((reinterpret_cast<uintptr_t>(node_tokens) | reinterpret_cast<uintptr_t>(choices) |
       reinterpret_cast<uintptr_t>(accepted_len) | reinterpret_cast<uintptr_t>(out_tokens)) & 3)
    return fail(VD_ERR_INVALID_ARG, "pointers must be 4-byte aligned");
  const vd_model_config& c = t->m->cfg;
  const Desc& d = t->d;
  TreeAcceptArgs a{};
  a.tokens = node_tokens ? node_tokens : d.base + d.tokens;
  a.choices = choices;
  a.parent = d.base + d.parent;
  a.cu_q = d.base + d.cu_q;
  a.cached_len = d.base + d.cached;
  a.page_table = d.base + d.page_table;
  a.pool = static_cast<__nv_bfloat16*>(pool->data);
  a.accepted_len = accepted_len;
  a.out_tokens = out_tokens;
  a.layer_elems = static_cast<long long>(pool->num_pages) * 2 * c.n_kv_heads * 16 * c.head_dim;
  a.B = d.B;
  a.layers = c.n_layers;
  a.Hkv = c.n_kv_heads;
  a.hd = c.head_dim;
  a.pt_stride = d.stride;
  a.out_stride = out_stride;
  a.status = t->m->status;
  return launch_tree_accept(a, s);
}

}  // extern "C"
