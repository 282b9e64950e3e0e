// The library's model and pool objects, shared by the translation units that
// implement the C ABI (api.cu, api_tree.cu).
#pragma once

#include <array>
#include <vector>

#include "vd_internal.h"

namespace vd {

constexpr int kSplitKeys = 512;  // S_kv, fixed for every model

struct ProfRec {
  int cls;
  int kernels;  // kernel launches between the two events
  cudaEvent_t a, b;
};
extern const char* const kKernelNames[];  // one name per KernelClass
enum KernelClass {
  K_EMBED, K_RMSNORM, K_GEMM_QKV, K_ROPE, K_ATTN, K_MERGE, K_GEMM_O, K_GEMM_GU, K_GEMM_DOWN, K_FINAL_NORM,
  K_GEMM_LM, K_SAMPLE, K_COUNT
};

// Activation buffer with TMA maps for row counts 1, 2, 4, ... (capped at
// the capacity), each in every token tile width: a GEMM over T rows uses the
// smallest row count covering T, so rows past T are either never fetched or
// (within the bucket) computed and discarded -- a GEMM column depends on its
// own row only.
struct ActBuf {
  __nv_bfloat16* ptr = nullptr;
  int cols = 0;
  std::vector<int> rows;
  std::vector<std::array<CUtensorMap, kNumBn>> maps;
  size_t bucket(int T) const {
    for (size_t i = 0; i < rows.size(); ++i)
      if (rows[i] >= T) return i;
    return rows.size() - 1;
  }
  ActMaps view(int T) const {
    ActMaps v;
    v.maps = maps[bucket(T)].data();
    v.rows = rows[bucket(T)];
    return v;
  }
};

// Host-side layout of the uploaded step descriptor (int32 offsets).
struct Desc {
  int T = 0, B = 0, R = 0, stride = 0;
  int tokens, positions, slot_page, cu_q, cached, page_table, logit_rows, dec_seq, dec_start, pre_seq, pre_start;
  // (merge_tok: offset of the token list the merge kernel folds)
  int n_dec = 0, n_pre = 0, items_dec = 0, items_pre = 0;
  bool fold = false;  // decode class in fold mode
  bool pre_tc = false;  // prefill class on the tcgen05 kernel (128 rows per CTA), else mma.sync (64)
  int merge_tok = 0, n_merge = 0;
  int grid_dec = 0, grid_pre = 0;  // attention CTAs launched (>= items; extra CTAs exit)
  int total = 0;
  const int* feed = nullptr;  // device tokens that entries -(1 + i) of `tokens` refer to
  const int* base = nullptr;  // device image the offsets above refer to
  // Token trees (vd_tree): the offsets of the tree's own arrays, and its split partials
  bool tree = false;
  int slots = 0, path = 0, path_off = 0, node_seq = 0, parent = 0;
  int blk_seq = 0, blk_first = 0, n_blk = 0, npg = 0, tail_rows = 0;  // blocks of nodes of the tail kernel
  // requests by the CTAs that run their shared tiles: 16, 32 or 64 rows on mma.sync, 128 on tcgen05
  struct {
    int seq = 0, start = 0, n = 0, items = 0;
  } cls[4];
  float *part_o = nullptr, *part_ml = nullptr;
  int part_splits = 0;  // splits per row of the partials
};

// What a captured step graph depends on beyond the model: every kernel
// argument and grid size of a step is a function of these fields.
struct GraphKey {
  unsigned long long pool_id = 0;
  const void* logits = nullptr;
  const void* tokens = nullptr;  // fused token choice (vd_step_sample) or null
  const void* feed = nullptr;    // device-side token feedback or null
  int T = 0, B = 0, R = 0, stride = 0, n_dec = 0, n_pre = 0, grid_dec = 0, grid_pre = 0, fold = 0, n_merge = 0;
  int pre_tc = 0;
  int fast = 0;
  unsigned plan_epoch = 0;  // GEMM plan override in force
  bool operator==(const GraphKey& o) const {
    return pool_id == o.pool_id && logits == o.logits && tokens == o.tokens && feed == o.feed && T == o.T && B == o.B && R == o.R && stride == o.stride &&
           n_dec == o.n_dec && n_pre == o.n_pre && grid_dec == o.grid_dec && grid_pre == o.grid_pre &&
           fold == o.fold && pre_tc == o.pre_tc && n_merge == o.n_merge && fast == o.fast &&
           plan_epoch == o.plan_epoch;
  }
};
struct GraphEntry {
  GraphKey key;
  cudaGraphExec_t exec = nullptr;
  long long used = 0;
};

}  // namespace vd

struct vd_model {
  vd_model_config cfg{};
  int device = 0;
  const __nv_bfloat16* embed = nullptr;
  const __nv_bfloat16* final_norm = nullptr;
  const __nv_bfloat16* lm_head = nullptr;
  std::vector<vd_layer_weights> layers;
  // fixed kernel choices
  int split = vd::kSplitKeys;
  int key_tile = 64;
  int max_splits = 0;
  int G = 1;
  // TMA maps
  std::vector<vd::WeightMaps> m_qkv, m_o, m_gu, m_down;
  vd::WeightMaps m_lm{};
  vd::ActBuf a, o, z, ar;
  // workspace
  __nv_bfloat16 *x = nullptr, *qkv = nullptr, *q = nullptr;
  __nv_bfloat16* hsub = nullptr;  // sandwich norms: a sub-layer's output before its norm
  float embed_scale = 0.f;        // 0: none, else bf16(sqrt(d)) as float
  int fold_mode = 0;              // 0: default (split mode), 1: fold the decode class whenever legal, 2: never
  int prefill_kernel = 0;         // 0: tcgen05 attention for the prefill class where hd allows, 1: mma.sync
  // fast (non-invariant) path: split-K for GEMMs with too few weight tiles
  int fast = 0;
  int n_sm = 0;
  float* splitk_part = nullptr;
  size_t splitk_cap = 0;          // floats
  std::vector<int> scratch_dec;   // host scratch of build_desc
  float gain_offset = 0.f;        // RMSNorm gains are w + gain_offset
  float *part_o = nullptr, *part_ml = nullptr;
  float *cos_g = nullptr, *sin_g = nullptr, *cos_l = nullptr, *sin_l = nullptr;
  vd::RopeShape rope_g{}, rope_l{};  // pair layout and rotated dims of global and local layers
  int* status = nullptr;
  int* d_desc = nullptr;
  int* h_desc[2] = {nullptr, nullptr};
  cudaEvent_t desc_ev[2] = {nullptr, nullptr};
  int desc_slot = 0;
  size_t desc_cap = 0;
  vd_sampler* d_samp = nullptr;
  float* samp_part_v = nullptr;  // per-chunk winners of the sampler's first pass
  int* samp_part_i = nullptr;
  float* fused_part_v = nullptr;  // per-32-row-group winners of the fused LM-head epilogue
  int* fused_part_i = nullptr;
  vd_sampler* h_samp = nullptr;
  void* filter_ws = nullptr;     // workspace of the filtered token choice (allocated on first use)
  cudaEvent_t samp_ev = nullptr;
  std::vector<void*> dev_allocs;
  // profiling
  bool profiling = false;
  std::vector<vd::ProfRec> recs;
  std::vector<cudaEvent_t> ev_pool;
  double prof_ms[vd::K_COUNT] = {};
  int prof_n[vd::K_COUNT] = {};
  int prof_k[vd::K_COUNT] = {};
  // graph replay of steps
  int graph_max = 0;
  cudaStream_t cap_stream = nullptr;
  std::vector<vd::GraphEntry> graphs;
  long long graph_clock = 0, graph_captures = 0, graph_replays = 0, graph_eager = 0;
};

struct vd_kv_pool {
  vd_model* m = nullptr;
  unsigned long long id = 0;  // never reused, unlike the host address
  int num_pages = 0;
  void* data = nullptr;
  bool owned = false;
  long long rows = 0;  // 16-slot rows of hd elements
  CUtensorMap map{};     // boxes for the mma.sync attention kernels
  CUtensorMap map_tc{};  // boxes for the tcgen05 attention kernel
};

namespace vd {

int check_model(const vd_model* m);
bool layer_is_local(const vd_model_config& c, int i);
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// cudaMalloc + clear, freed with the model.
int dev_alloc(vd_model* m, void** p, size_t bytes);
// The kernel sequence of one step whose descriptor is at d.base.
int enqueue_step(vd_model* m, vd_kv_pool* pool, const Desc& d, float* logits_out, int* tokens_out, cudaStream_t s);
void drop_graphs(vd_model* m);
int run_rope(vd_model* m, vd_kv_pool* pool, int layer, const Desc& d, const __nv_bfloat16* qkv, __nv_bfloat16* q_out,
             cudaStream_t s);
// Attention and RoPE + K/V write of a token tree (api_tree.cu).
int run_tree_attention(vd_model* m, vd_kv_pool* pool, int layer, const Desc& d, const __nv_bfloat16* q,
                       __nv_bfloat16* out, cudaStream_t s);

// ---------------------------------------------------------------- profiling
inline cudaEvent_t take_event(vd_model* m) {
  if (!m->ev_pool.empty()) {
    cudaEvent_t e = m->ev_pool.back();
    m->ev_pool.pop_back();
    return e;
  }
  cudaEvent_t e = nullptr;
  cudaEventCreate(&e);
  return e;
}
struct Prof {
  vd_model* m;
  int cls;
  cudaStream_t s;
  cudaEvent_t a = nullptr;
  int kernels = 1;
  Prof(vd_model* m_, int cls_, cudaStream_t s_) : m(m_), cls(cls_), s(s_) {
    if (m->profiling) {
      a = take_event(m);
      cudaEventRecord(a, s);
    }
  }
  ~Prof() {
    if (m->profiling) {
      cudaEvent_t b = take_event(m);
      cudaEventRecord(b, s);
      m->recs.push_back({cls, kernels, a, b});
    }
  }
};

}  // namespace vd
