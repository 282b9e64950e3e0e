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
// layout of a TMA-staged tile.  For trees whose tail does not fit shared memory
// (below); bound by the latency of its gathers.
constexpr int kTailWarps = 4;

// Whether a bounded wait of this step has given up; one read for the whole
// CTA keeps its exit uniform.
__device__ __forceinline__ bool skip_step(int* status) {
  __shared__ int skip;
  if (threadIdx.x == 0) skip = status ? *reinterpret_cast<volatile int*>(status) : 0;
  __syncthreads();
  return skip != 0;
}


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
  if (skip_step(a.status)) return;
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
    // the pool row of key key0 + lane: a cached slot, or the slot of the path's node at that position (those below the
    // window too: the decoded path's products take them, with the weight 0)
    const int key = key0 + lane;
    long long row = -1;
    if (key <= p) {
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

// The same with the rows staged once per CTA, for trees whose tail fits shared
// memory.  A CTA owns a block of nodes of one (request, KV head) and copies the
// cached keys past the shared tiles and every node's K and V into rows of its
// own (16-byte chunks swizzled within 128 bytes).  A warp (DS of them, each with
// its part of the head dimension) folds up to 16 / G nodes at once, their query
// heads as the 16 rows of an mma tile: scores and P V are one chain of
// instructions per node, on K and V rows gathered by ldmatrix address from the
// node's path, with the other nodes' rows ignored in the scores and zero in P
// (they add nothing to O); softmax, rescale and state are shared.  16-key
// halves of a tile in which a node sees no key are left out: zeros again.  A zero
// of P times an infinity or NaN of V is no zero, so a node's masked keys take a
// staged row of zeros, and a CTA that finds such a value among its V rows (each
// thread in what it copied) folds its nodes one after the other, each on the
// state it started from.
// Bound by its chains' latency at two CTAs of four warps per SM (210 registers:
// Q, the state and the scores of 16 rows; three CTAs spill and measured the
// same): at 32 trees x 64 nodes x 8 KV heads, 4 rows each, 51 us, a quarter of
// the mma.sync rate, 11 M warp instructions.  One node per warp took 85 us.  The
// look for values that are not finite takes 0.1 % of the operator there (0.5 us of
// 12.5 for 24 trees of 9 nodes without a shared tile).
template <int HD>
struct Staged {
  static constexpr int ROW = HD * 2;  // bytes of a K or V row
  // K rows, V rows, and a V row of zeros
  static constexpr size_t bytes(int tail_rows) { return 128 + (static_cast<size_t>(tail_rows) * 2 + 1) * ROW; }
  __device__ static __forceinline__ uint32_t off(int row, int chunk) {
    return row * ROW + ((chunk & ~7) << 4) + (((chunk & 7) ^ (row & 7)) << 4);
  }
};
constexpr size_t kStagedBytes = 100 * 1024;  // two CTAs share an SM

// Whether one of the two bf16 is an infinity or NaN (exponent all ones: adding
// its lowest bit carries into the sign's place).
__device__ __forceinline__ uint32_t not_finite(uint32_t two) {
  return ((two & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}

// A warp's part of a staged tail: the nodes [first, first + count) of one request
// and KV head, dims [dim0, dim0 + ND).
template <int HD, int DS>
struct TailFold {
  using S = Staged<HD>;
  static constexpr int BNK = 32, ND = HD / DS;
  int kvh, nodes, c, first, count, shared, rows, dim0;
  const int* table;
  uint32_t sk, sv;
  int node[2], pos[2], lo[2];
  bool valid[2];
  size_t out_row[2];  // of the row in q, and times max_splits in the partials
  int p_max, lo_min;
  int my_p, my_path;  // lane n of the warp knows node n
  uint32_t qf[HD / 16][4];
  RowState<ND> st;

  // The description was written before the step's first kernel.
  __device__ __forceinline__ void init(const TreeTailArgs& a, uint32_t smem) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, item = blockIdx.x;
    const int b = a.blk_seq[item], n0 = a.cu_q[b], G = a.Hq / a.Hkv;
    kvh = blockIdx.y;
    nodes = a.cu_q[b + 1] - n0;
    c = a.cached_len[b];
    first = a.blk_first[item] + (warp / DS) * a.npg;
    count = max(0, min(a.npg, nodes - first));
    table = a.page_table + static_cast<size_t>(b) * a.pt_stride;
    shared = c / BNK * BNK;
    rows = c - shared + nodes;  // staged row i: slot shared + i
    dim0 = (warp % DS) * ND;
    sk = smem;
    sv = sk + rows * S::ROW;
    p_max = -1;
    lo_min = INT_MAX;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = (lane >> 2) + 8 * r;
      node[r] = i / G;
      valid[r] = node[r] < count;
      const int t = n0 + first + (valid[r] ? node[r] : 0);
      const int p = valid[r] ? a.positions[t] : -1;
      pos[r] = p;
      lo[r] = valid[r] ? (a.window > 0 ? max(0, p - a.window + 1) : 0) : 1;
      out_row[r] = static_cast<size_t>(t) * a.Hq + kvh * G + i % G;
      p_max = max(p_max, p);
      if (valid[r]) lo_min = min(lo_min, lo[r]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      p_max = max(p_max, __shfl_xor_sync(0xffffffffu, p_max, o));
      lo_min = min(lo_min, __shfl_xor_sync(0xffffffffu, lo_min, o));
    }
    const int my_t = n0 + first + min(lane, max(count - 1, 0));
    my_p = lane < count ? a.positions[my_t] : -1;
    my_path = lane < count ? a.path_off[my_t] : 0;
  }
  __device__ __forceinline__ void load_q(const TreeTailArgs& a) {
    const int t4 = threadIdx.x & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const __nv_bfloat16* qr = a.q + out_row[r] * HD;
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        qf[kk][r] = valid[r] ? *reinterpret_cast<const uint32_t*>(qr + kk * 16 + t4 * 2) : 0u;
        qf[kk][2 + r] = valid[r] ? *reinterpret_cast<const uint32_t*>(qr + kk * 16 + 8 + t4 * 2) : 0u;
      }
    }
  }
  // The state of the split that the shared tiles began: m and l (of every warp of a
  // node; ML) and the O of this warp's columns (which no other warp writes).  One
  // condition for all of a row's loads (asked beside each of them, a tree of 8 nodes
  // took 18.5 us, and 17.1 so).
  template <bool ML>
  __device__ __forceinline__ void load_state(const TreeTailArgs& a) {
    const int t4 = threadIdx.x & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool begun = valid[r] && max(lo[r], shared / a.split * a.split) < shared;
      const size_t at = out_row[r] * a.max_splits + shared / a.split;
      if constexpr (ML) {
        st.m[r] = begun ? a.part_ml[at * 2] : -INFINITY;
        st.l[r] = begun ? a.part_ml[at * 2 + 1] : 0.f;
      }
      const float* po = a.part_o + at * HD + dim0;
#pragma unroll
      for (int n = 0; n < ND / 8; ++n) {
        const float2 v = begun ? *reinterpret_cast<const float2*>(po + n * 8 + t4 * 2) : make_float2(0.f, 0.f);
        st.o[n][2 * r] = v.x;
        st.o[n][2 * r + 1] = v.y;
      }
    }
  }
  __device__ __forceinline__ void store(const TreeTailArgs& a, int r, int split) {
    const int t4 = threadIdx.x & 3;
    const size_t at = out_row[r] * a.max_splits + split;
    if (t4 == 0 && dim0 == 0) {
      a.part_ml[at * 2] = st.m[r];
      a.part_ml[at * 2 + 1] = st.l[r];
    }
    float* po = a.part_o + at * HD + dim0;
#pragma unroll
    for (int n = 0; n < ND / 8; ++n)
      *reinterpret_cast<float2*>(po + n * 8 + t4 * 2) = make_float2(st.o[n][2 * r], st.o[n][2 * r + 1]);
  }

  // Folds the tail of the warp's nodes, or APART that of node `only`, and stores
  // its splits.  row_s: a tile's staged rows, of each node.
  template <bool APART>
  __device__ __forceinline__ void fold(const TreeTailArgs& a, int (*row_s)[BNK], int only) {
    const int lane = threadIdx.x & 31, mi = lane >> 3, r8 = lane & 7;
    const int na = APART ? only : 0, nb = APART ? only + 1 : count;
    auto mine = [&](int r) { return APART ? valid[r] && node[r] == only : valid[r]; };
    int key0 = max(shared, lo_min / BNK * BNK);
    for (; key0 <= p_max; key0 += BNK) {
      if (key0 != shared && key0 % a.split == 0) {  // the previous split is complete
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (mine(r) && max(lo[r], key0 - a.split) <= min(pos[r], key0 - 1)) store(a, r, key0 / a.split - 1);
          st.m[r] = -INFINITY;
          st.l[r] = 0.f;
        }
#pragma unroll
        for (int n = 0; n < ND / 8; ++n) st.o[n][0] = st.o[n][1] = st.o[n][2] = st.o[n][3] = 0.f;
      }
      // tiles that are none of node n's: past its position, or (where it matters) below its window
      auto skips = [&](int p) { return p < key0 || (APART && a.window > 0 && p - a.window + 1 >= key0 + BNK); };
      // ---- scores: each node's on its own keys
      float s[BNK / 8][4];
#pragma unroll
      for (int j = 0; j < BNK / 8; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
      // the row of each node's key at key0 + lane: a cached slot's, that of the path's node at that position, or past
      // the node's own the row of zeros (as a K row, whatever lies there: masked)
      const int key = key0 + lane;
      __syncwarp();
#pragma unroll 4
      for (int n = na; n < nb; ++n) {
        const int p = __shfl_sync(0xffffffffu, my_p, n), path = __shfl_sync(0xffffffffu, my_path, n);
        row_s[n][lane] = key < c ? key - shared : c - shared + (key <= p ? a.path[path + key - c] : nodes);
      }
      __syncwarp();
      for (int n = na; n < nb; ++n) {
        const int p = __shfl_sync(0xffffffffu, my_p, n);
        if (skips(p)) continue;
        const bool both = p >= key0 + 16;
#pragma unroll
        for (int jp = 0; jp < BNK / 16; ++jp) {
          if (jp == 1 && !both) continue;
          const int kr = row_s[n][jp * 16 + (mi >> 1) * 8 + r8];
          float x[2][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[0][e] = x[1][e] = 0.f;
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            uint32_t f[4];
            ldmatrix_x4(f, sk + S::off(kr, kk * 2 + (mi & 1)));
            mma_bf16_16816(x[0], qf[kk], f);
            mma_bf16_16816(x[1], qf[kk], f + 2);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[2 * jp + j][e] = node[e >> 1] == n ? x[j][e] : s[2 * jp + j][e];
        }
      }
      // ---- softmax of the tile, all rows
      float mx[2], mnew[2], alpha[2], rs[2];
      bool rv[2];
      uint32_t pa[BNK / 16][4], pl[BNK / 16][4];
      tile_mask_max<BNK, false>(s, mx, key0, pos, lo, a.scale_log2, lane);
#pragma unroll
      for (int r = 0; r < 2; ++r) tile_running_max(st.m[r], mx[r], mnew[r], alpha[r], rv[r]);
      tile_probs<BNK, false>(s, mnew, pa, pl, rs);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        tile_update_l(st.l[r], alpha[r], rs[r], rv[r]);
        st.m[r] = mnew[r];
      }
      tile_rescale<ND, false>(st.o, alpha);
      // ---- P V: each node's rows of P on its own values
      for (int n = na; n < nb; ++n) {
        const int p = __shfl_sync(0xffffffffu, my_p, n);
        if (skips(p)) continue;
        const bool both = p >= key0 + 16;
#pragma unroll
        for (int ks = 0; ks < BNK / 16; ++ks) {
          if (ks == 1 && !both) continue;
          const int vr = row_s[n][ks * 16 + (mi & 1) * 8 + r8];
          uint32_t ph[4], pw[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ph[e] = node[e & 1] == n ? pa[ks][e] : 0u;
            pw[e] = node[e & 1] == n ? pl[ks][e] : 0u;
          }
#pragma unroll
          for (int np = 0; np < ND / 16; ++np) {
            uint32_t f[4];
            ldmatrix_x4_trans(f, sv + S::off(vr, dim0 / 8 + np * 2 + (mi >> 1)));
            mma_bf16_16816(st.o[2 * np], ph, f);
            mma_bf16_16816(st.o[2 * np], pw, f);
            mma_bf16_16816(st.o[2 * np + 1], ph, f + 2);
            mma_bf16_16816(st.o[2 * np + 1], pw, f + 2);
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)  // rows whose last split is the one just folded (the others' are stored)
      if (mine(r) && pos[r] / a.split == (key0 - BNK) / a.split) store(a, r, pos[r] / a.split);
  }
};

// The nodes one after the other, each on the state it starts from (ml: m and l,
// read before any warp of the node stored one).  Out of line: its copy of the fold
// costs the usual one no registers.
template <int HD, int DS>
__device__ __noinline__ void fold_apart(const TreeTailArgs& a, uint32_t smem, int (*row_s)[32], float4 ml) {
  TailFold<HD, DS> f;
  f.init(a, smem);
  f.load_q(a);
#pragma unroll 1
  for (int n = 0; n < f.count; ++n) {
    f.st.m[0] = ml.x;
    f.st.m[1] = ml.y;
    f.st.l[0] = ml.z;
    f.st.l[1] = ml.w;
    f.template load_state<false>(a);
    f.template fold<true>(a, row_s, n);
  }
}

// MANY: a warp folds more than one node, and looks for values that are not finite
// (with one node to a warp there is nobody to keep them from, and the look cost a
// tree of 8 nodes 0.5 of its 17.1 us).
template <int HD, int DS, bool MANY>
__global__ void __launch_bounds__(kTailWarps * 32, 2) tree_tail_staged_kernel(const __grid_constant__ TreeTailArgs a) {
  using S = Staged<HD>;
  constexpr int BNK = 32, CH = HD / 8;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int row_s[kTailWarps][16][BNK];
  if (skip_step(a.status)) return;
  uint8_t* smem = smem_raw + ((128 - (smem_u32(smem_raw) & 127)) & 127);
  TailFold<HD, DS> f;
  f.init(a, smem_u32(smem));
  uint8_t* vrows = smem + f.rows * S::ROW;
  if (!a.early) pdl_wait();
  for (int i = threadIdx.x; i < f.rows * CH; i += kTailWarps * 32) {
    const int r = i / CH, ch = i % CH, slot = f.shared + r;
    const size_t row = (static_cast<size_t>(f.table[slot >> 4]) * 2 * a.Hkv + f.kvh) * 16 + (slot & 15);
    const __nv_bfloat16* src = a.pool + row * HD + ch * 8;
    cp_async16(smem + S::off(r, ch), src);
    cp_async16(vrows + S::off(r, ch), src + static_cast<size_t>(a.Hkv) * 16 * HD);
  }
  if (threadIdx.x < CH)
    *reinterpret_cast<uint4*>(vrows + S::off(f.rows, threadIdx.x)) = make_uint4(0u, 0u, 0u, 0u);
  f.load_q(a);
  if (a.early) pdl_wait();
  pdl_trigger();
  f.template load_state<true>(a);
  cp_async_wait_all();
  int(*rows_of)[BNK] = row_s[threadIdx.x >> 5];
  // the rows have landed, and every warp of a node has its m and l before one stores another
  if constexpr (MANY) {
    uint32_t sick = 0;
    for (int i = threadIdx.x; i < f.rows * CH; i += kTailWarps * 32) {
      const uint4 v = *reinterpret_cast<const uint4*>(vrows + S::off(i / CH, i % CH));
      sick |= not_finite(v.x) | not_finite(v.y) | not_finite(v.z) | not_finite(v.w);
    }
    if (__syncthreads_or(sick != 0)) {
      fold_apart<HD, DS>(a, smem_u32(smem), rows_of, make_float4(f.st.m[0], f.st.m[1], f.st.l[0], f.st.l[1]));
      return;
    }
  } else {
    __syncthreads();
  }
  if (f.count > 0) f.template fold<false>(a, rows_of, 0);
}

template <int HD>
int launch_tail_staged(const TreeTailArgs& a, cudaStream_t s) {
  constexpr int DS = HD == 256 ? 2 : 1;
  const size_t smem = Staged<HD>::bytes(a.tail_rows);
  auto k = a.npg > 1 ? tree_tail_staged_kernel<HD, DS, true> : tree_tail_staged_kernel<HD, DS, false>;
  // the most that any launch takes: another thread's may come between this and the launch
  VD_CUDA_TRY(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kStagedBytes)));
  VD_CUDA_TRY(launch_k(k, dim3(a.n_blk, a.Hkv), dim3(kTailWarps * 32), smem, s, a));
  return VD_OK;
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
// A path longer than out_stride ends there.
// Every layer's CTA finds the path for itself (no second launch), then moves
// the K/V of the path's node at depth d from slot c + node to slot c + d.  A
// thread moves the same 16-byte column of every node, in ascending depth: a
// node's number is at least its depth, so no slot is overwritten before it
// has been read.  Bound by one chain of dependent reads (parents and tokens, the
// path's pages, K/V), whatever the batch: 5.7 us for 32 trees of 32 nodes in 32
// layers of 8 heads x 128 (33 MB moved if half of 8-node chains are accepted),
// the same for one tree of 8.
constexpr int kAcceptThreads = 256;
constexpr int kAcceptBatch = 8;  // nodes read before their copies are written

__global__ void __launch_bounds__(kAcceptThreads) tree_accept_kernel(TreeAcceptArgs a) {
  extern __shared__ int next[];  // [nodes] the child the path goes on to, then the path itself
  if (skip_step(a.status)) return;
  const int b = blockIdx.x, layer = blockIdx.y;
  const int n0 = a.cu_q[b], n = a.cu_q[b + 1] - n0, c = a.cached_len[b];
  int* path = next + n;
  __shared__ int length;
  for (int i = threadIdx.x; i < n; i += kAcceptThreads) next[i] = INT_MAX;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i < n; i += kAcceptThreads) {
    const int p = a.parent[n0 + i];
    if (p >= 0 && a.tokens[n0 + i] == a.choices[n0 + p]) atomicMin(&next[p], i);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int len = 0;
    for (int i = 0; i != INT_MAX && len < a.out_stride; i = next[i]) path[len++] = i;
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

// Nodes that a warp folds at once: one while the launch has warps to spare (a
// node's chains are then the latency: 7 us for 8 nodes), up to 16 / G where it
// has not (32 x 64 nodes: 51 us, against 85 us of one per warp).  0: the tail
// does not fit.
int tree_nodes_per_warp(int hd, int nodes, int Hkv, int G, int tail_rows, int n_sm, int* blk_nodes) {
  const size_t bytes = hd == 64 ? Staged<64>::bytes(tail_rows)
                       : hd == 128 ? Staged<128>::bytes(tail_rows) : Staged<256>::bytes(tail_rows);
  *blk_nodes = 1;
  if (bytes > kStagedBytes) return 0;
  const int groups = kTailWarps / (hd == 256 ? 2 : 1);
  const long long each = (static_cast<long long>(nodes) * Hkv - 1) / (2LL * n_sm * groups) + 1;
  const int npg = static_cast<int>(each < 16 / G ? each : 16 / G);
  *blk_nodes = groups * npg;
  return npg;
}

int launch_tree_tail(const TreeTailArgs& a, int hd, cudaStream_t s) {
  if (a.T <= 0) return VD_OK;
  if (a.npg > 0) {
    if (hd == 64) return launch_tail_staged<64>(a, s);
    if (hd == 128) return launch_tail_staged<128>(a, s);
    if (hd == 256) return launch_tail_staged<256>(a, s);
  }
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
