// Token trees over the paged cache: the key tiles that differ from node to
// node, and the acceptance of a path.
//
// A request's tree hangs below its cached_len = c cached tokens.  Node i has
// its K/V in slot c + i and stands at position p = c + depth(i); it sees the
// cached keys and, at positions c .. p, the nodes of its path.  Decoding that
// path token by token would fold the key tiles [32 t, 32 t + 31] of the
// positions 0 .. p in ascending order, cut into splits; that is the order a
// node's row follows here too, so its result is that of the decoded path, bit
// for bit.  The tiles below c rounded down to a tile hold the same keys for
// every node: the kernels of attention.cu and attention_tc.cu fold them with
// all nodes as rows, and leave a split partial (m, l, O), which is exactly
// the online-softmax state after the last of those tiles.  The tail kernel
// takes that state up.
#include <limits.h>

#include "attn_tile.cuh"
#include "vd_device.cuh"
#include "vd_internal.h"

namespace vd {
namespace {

// A group of DS warps folds the tail tiles of one (node, KV head): the
// group's query heads are the first G of the 16 rows of the mma tile, and its
// keys are gathered from the slots of its path, 16 bytes per copy, into the
// layout of a TMA-staged tile.
constexpr int kTailWarps = 4;

template <int HD, int DS>
__global__ void __launch_bounds__(kTailWarps * 32) tree_tail_kernel(TreeTailArgs a) {
  using C = AttnCfg<HD>;
  constexpr int ND = HD / DS, GROUPS = kTailWarps / DS, CH = HD / 8;  // CH: 16-byte chunks of a row
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / DS, part = warp % DS, gl = part * 32 + lane;
  uint8_t* sk = smem + group * 2 * C::TILE_BYTES;
  uint8_t* sv = sk + C::TILE_BYTES;
  auto group_sync = [&] {
    if constexpr (DS == 1) __syncwarp();
    else asm volatile("barrier.sync %0, %1;" ::"r"(1 + group), "r"(DS * 32) : "memory");  // not .aligned: per thread
  };
  // the tree's description was written before the step's first kernel
  const int item = blockIdx.x * GROUPS + group;
  if (item >= a.T * a.Hkv) return;
  const int t = item / a.Hkv, kvh = item % a.Hkv;
  const int b = a.node_seq[t], c = a.cached_len[b], p = a.positions[t], node0 = a.path_off[t];
  const int* table = a.page_table + static_cast<size_t>(b) * a.pt_stride;
  const int lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
  const int shared = c / C::BNK * C::BNK;
  pdl_wait();
  pdl_trigger();
  if (a.status && *reinterpret_cast<volatile int*>(a.status)) return;  // the same for the whole group

  const int G = a.Hq / a.Hkv, gq = lane >> 2, t4 = lane & 3, dim0 = part * ND;
  const bool lower8 = G <= 8;
  int pos[2], low[2];
  bool valid[2];
  uint32_t qf[HD / 16][4];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int h = gq + 8 * r;
    valid[r] = h < G;
    pos[r] = valid[r] ? p : -1;
    low[r] = valid[r] ? lo : 1;
    const __nv_bfloat16* qr = a.q + (static_cast<size_t>(t) * a.Hq + kvh * G + (valid[r] ? h : 0)) * HD;
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
      qf[kk][r] = valid[r] ? *reinterpret_cast<const uint32_t*>(qr + kk * 16 + t4 * 2) : 0u;
      qf[kk][2 + r] = valid[r] ? *reinterpret_cast<const uint32_t*>(qr + kk * 16 + 8 + t4 * 2) : 0u;
    }
  }
  RowState<ND> st;
  auto base = [&](int r, int split) {
    return (static_cast<size_t>(t) * a.Hq + kvh * G + gq + 8 * r) * a.max_splits + split;
  };
  auto clear = [&] {
    st.m[0] = st.m[1] = -INFINITY;
    st.l[0] = st.l[1] = 0.f;
#pragma unroll
    for (int n = 0; n < ND / 8; ++n) st.o[n][0] = st.o[n][1] = st.o[n][2] = st.o[n][3] = 0.f;
  };
  auto store = [&](int split) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (!valid[r]) continue;
      const size_t at = base(r, split);
      if (t4 == 0 && part == 0) {
        a.part_ml[at * 2] = st.m[r];
        a.part_ml[at * 2 + 1] = st.l[r];
      }
      float* po = a.part_o + at * HD + dim0;
#pragma unroll
      for (int n = 0; n < ND / 8; ++n)
        *reinterpret_cast<float2*>(po + n * 8 + t4 * 2) = make_float2(st.o[n][2 * r], st.o[n][2 * r + 1]);
    }
  };
  clear();
  if (max(lo, shared / a.split * a.split) < shared) {  // the split was begun by the shared tiles
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (!valid[r]) continue;
      const size_t at = base(r, shared / a.split);
      st.m[r] = a.part_ml[at * 2];
      st.l[r] = a.part_ml[at * 2 + 1];
      const float* po = a.part_o + at * HD + dim0;
#pragma unroll
      for (int n = 0; n < ND / 8; ++n) {
        const float2 v = *reinterpret_cast<const float2*>(po + n * 8 + t4 * 2);
        st.o[n][2 * r] = v.x;
        st.o[n][2 * r + 1] = v.y;
      }
    }
  }
  for (int key0 = max(shared, lo / C::BNK * C::BNK); key0 <= p; key0 += C::BNK) {
    if (key0 != shared && key0 % a.split == 0) {  // the previous split is complete
      if (max(lo, key0 - a.split) < key0) store(key0 / a.split - 1);
      clear();
    }
    // the pool row of key key0 + lane: a cached slot, or the slot of the path's node at that position
    const int key = key0 + lane;
    long long row = -1;
    if (key >= lo && key <= p) {
      const int slot = key < c ? key : c + a.path[node0 + key - c];
      row = (static_cast<long long>(table[slot >> 4]) * 2 * a.Hkv + kvh) * 16 + (slot & 15);
    }
    group_sync();  // the previous tile has been read
#pragma unroll 4
    for (int i = gl; i < C::BNK * CH; i += DS * 32) {
      const int k = i / CH, ch = i % CH;
      const long long rk = __shfl_sync(0xffffffffu, row, k);
      const uint32_t off = kv_off<HD>(k, ch);
      if (rk >= 0) {
        const __nv_bfloat16* src = a.pool + rk * HD + ch * 8;
        cp_async16(sk + off, src);
        cp_async16(sv + off, src + static_cast<long long>(a.Hkv) * 16 * HD);
      } else {
        *reinterpret_cast<uint4*>(sk + off) = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(sv + off) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    cp_async_wait_all();
    group_sync();
    if (lower8)
      attn_tile<HD, C::BNK, ND, true>(st, qf, smem_u32(sk), smem_u32(sv), key0, pos, low, a.scale_log2, lane, dim0);
    else
      attn_tile<HD, C::BNK, ND, false>(st, qf, smem_u32(sk), smem_u32(sv), key0, pos, low, a.scale_log2, lane, dim0);
  }
  store(p / a.split);
}

template <int HD, int DS>
int launch_tail_t(const TreeTailArgs& a, cudaStream_t s) {
  using C = AttnCfg<HD>;
  constexpr int kGroups = kTailWarps / DS, kSmem = 1024 + kGroups * 2 * C::TILE_BYTES;
  VD_CUDA_TRY(cudaFuncSetAttribute(tree_tail_kernel<HD, DS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
  const int items = a.T * a.Hkv;
  VD_CUDA_TRY(launch_k(tree_tail_kernel<HD, DS>, dim3((items + kGroups - 1) / kGroups), dim3(kTailWarps * 32), kSmem, s,
                       a));
  return VD_OK;
}

// Acceptance.  CTA (request, layer): from the root, the path goes on to the
// lowest-numbered child that holds the token chosen after its last node.
// Every layer's CTA finds the path for itself (no second launch), then moves
// the K/V of the path's node at depth d from slot c + node to slot c + d.  A
// thread moves the same 16-byte column of every node, in ascending depth: a
// node's number is at least its depth, so no slot is overwritten before it
// has been read.
constexpr int kAcceptThreads = 256;
constexpr int kAcceptBatch = 8;  // nodes read before their copies are written

__global__ void __launch_bounds__(kAcceptThreads) tree_accept_kernel(TreeAcceptArgs a) {
  extern __shared__ int next[];  // [nodes] the child the path goes on to, then the path itself
  const int b = blockIdx.x, layer = blockIdx.y;
  const int n0 = a.cu_q[b], n = a.cu_q[b + 1] - n0, c = a.cached_len[b];
  int* path = next + n;
  __shared__ int length;
  for (int i = threadIdx.x; i < n; i += kAcceptThreads) next[i] = INT_MAX;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  if (a.status && *reinterpret_cast<volatile int*>(a.status)) return;
  for (int i = threadIdx.x; i < n; i += kAcceptThreads) {
    const int p = a.parent[n0 + i];
    if (p >= 0 && a.tokens[n0 + i] == a.choices[n0 + p]) atomicMin(&next[p], i);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int len = 0;
    for (int i = 0; i != INT_MAX; i = next[i]) path[len++] = i;
    length = len;
  }
  __syncthreads();
  const int len = length;
  if (layer == 0) {
    if (threadIdx.x == 0) a.accepted_len[b] = len;
    for (int d = threadIdx.x; d < a.out_stride; d += kAcceptThreads)
      a.out_tokens[static_cast<size_t>(b) * a.out_stride + d] = d < len ? a.choices[n0 + path[d]] : -1;
  }
  const int cols = 2 * a.Hkv * a.hd / 8, row8 = a.hd / 8;
  const int* table = a.page_table + static_cast<size_t>(b) * a.pt_stride;
  uint4* pool = reinterpret_cast<uint4*>(a.pool + layer * a.layer_elems);
  for (int col = threadIdx.x; col < cols; col += kAcceptThreads) {
    const int kvg = col / row8, ch = col % row8;  // (K or V, head), chunk
    auto at = [&](int slot) {
      return ((static_cast<size_t>(table[slot >> 4]) * 2 * a.Hkv + kvg) * 16 + (slot & 15)) * row8 + ch;
    };
    for (int d0 = 1; d0 < len; d0 += kAcceptBatch) {
      uint4 v[kAcceptBatch];
#pragma unroll
      for (int k = 0; k < kAcceptBatch; ++k)
        if (d0 + k < len && path[d0 + k] != d0 + k) v[k] = pool[at(c + path[d0 + k])];
#pragma unroll
      for (int k = 0; k < kAcceptBatch; ++k)
        if (d0 + k < len && path[d0 + k] != d0 + k) pool[at(c + d0 + k)] = v[k];
    }
  }
}

}  // namespace

int launch_tree_tail(const TreeTailArgs& a, int hd, cudaStream_t s) {
  if (a.T <= 0) return VD_OK;
  if (hd == 64) return launch_tail_t<64, 1>(a, s);
  if (hd == 128) return launch_tail_t<128, 1>(a, s);
  if (hd == 256) return launch_tail_t<256, 2>(a, s);
  return fail(VD_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
}

int launch_tree_accept(const TreeAcceptArgs& a, cudaStream_t s) {
  if (a.B <= 0) return VD_OK;
  VD_CUDA_TRY(launch_k(tree_accept_kernel, dim3(a.B, a.layers), dim3(kAcceptThreads),
                       2 * static_cast<size_t>(kTreeMaxNodes) * sizeof(int), s, a));
  return VD_OK;
}

}  // namespace vd
