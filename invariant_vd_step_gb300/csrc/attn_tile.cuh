// The per-tile steps of the mma.sync attention kernels (attention.cu) and of
// the tree-tail kernel (tree.cu): scores, masking, online softmax and P V of
// one 32-key tile for the 16 rows of a warp.
#pragma once

#include <math.h>

#include "vd_device.cuh"

namespace vd {

template <int HD>
struct AttnCfg {
  static constexpr int BNK = 32;                     // keys per tile
  static constexpr int PAGES = BNK / 16;             // 16-token pages per tile
  static constexpr int PAGE_BYTES = 16 * HD * 2;     // one page of one KV head
  static constexpr int TILE_BYTES = BNK * HD * 2;
  static constexpr int MAX_STAGES = 8;
  static constexpr int PIDS = 64;  // page ids a decode CTA stages: every page of its split
  static constexpr int STATIC_SMEM = PIDS * 4 + 16;
  // K + V tiles of `stages` pipeline stages, their barriers, the abort flag
  static constexpr int smem(int stages) { return 1024 + stages * 2 * TILE_BYTES + MAX_STAGES * 8 + 16; }
};

// Byte offset of (key, 16-byte chunk along hd) inside a K or V tile staged
// by the 3-D TMA box (64, hd/64, 16) with the 128-byte swizzle.
template <int HD>
__device__ __forceinline__ uint32_t kv_off(int key, int chunk) {
  const int pg = key >> 4, slot = key & 15;
  const int lr = slot * (HD / 64) + (chunk >> 3);
  return pg * AttnCfg<HD>::PAGE_BYTES + lr * 128 + (((chunk & 7) ^ (lr & 7)) << 4);
}

template <int ND>
struct RowState {
  float m[2], l[2];     // rows g and g+8 of the warp
  float o[ND / 8][4];   // mma C fragments of the ND output dims this warp owns
};

// The steps of one key tile for the 16 rows of a warp (rows g and g + 8 of
// lane (g, t4)).  `attn_tile` runs them back to back, one tile at a time;
// the scores-first decode kernel runs the same steps over a whole split in
// three phases.  Either way every row's values pass through the same
// operations in the same order.  LOWER8: rows 8..15 of the warp are known
// to hold no row (a decode CTA of at most 8 rows), so their masking,
// softmax and rescale are skipped: their weights are exactly 0 either way,
// and the other rows' instructions are unchanged.

// S = Q K^T of a 32-key tile: per 8-key block, HD/16 K = 16 steps from zero.
template <int HD, int BNK>
__device__ __forceinline__ void tile_scores(float (&s)[BNK / 8][4], const uint32_t (&qf)[HD / 16][4], uint32_t kbase,
                                            int lane) {
  const int mi = lane >> 3, r8 = lane & 7;
#pragma unroll
  for (int j = 0; j < BNK / 8; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
  for (int kk = 0; kk < HD / 16; ++kk) {
#pragma unroll
    for (int jp = 0; jp < BNK / 16; ++jp) {
      uint32_t b[4];
      ldmatrix_x4(b, kbase + kv_off<HD>(jp * 16 + (mi >> 1) * 8 + r8, kk * 2 + (mi & 1)));
      mma_bf16_16816(s[2 * jp], qf[kk], b);
      mma_bf16_16816(s[2 * jp + 1], qf[kk], b + 2);
    }
  }
}

// Scores to the log2 domain, -inf outside each row's keys [lo, pos]; the
// tile's maximum of rows g and g + 8 over the lane quad.
template <int BNK, bool LOWER8>
__device__ __forceinline__ void tile_mask_max(float (&s)[BNK / 8][4], float (&mx)[2], int key0, const int (&pos)[2],
                                              const int (&lo)[2], float scale_log2, int lane) {
  const int t4 = lane & 3;
  mx[0] = mx[1] = -INFINITY;
#pragma unroll
  for (int j = 0; j < BNK / 8; ++j) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = e >> 1;
      if (LOWER8 && r == 1) {
        s[j][e] = -INFINITY;
        continue;
      }
      const int key = key0 + j * 8 + t4 * 2 + (e & 1);
      const bool vis = key >= lo[r] && key <= pos[r];
      const float v = vis ? __fmul_rn(s[j][e], scale_log2) : -INFINITY;
      s[j][e] = v;
      mx[r] = fmaxf(mx[r], v);
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    if (LOWER8 && r == 1) continue;  // stays -inf: the row keeps its state
    mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
    mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
  }
}

// The running maximum after a tile with row maximum mx, the factor that
// rescales the state before it, and whether the row saw a key in it (a row
// that saw none keeps its state bit for bit: alpha = 1, m unchanged).
__device__ __forceinline__ void tile_running_max(float m, float mx, float& mnew, float& alpha, bool& rv) {
  rv = mx != -INFINITY;
  mnew = rv ? fmaxf(m, mx) : m;
  alpha = rv ? ex2(__fsub_rn(m, mnew)) : 1.0f;
}

// P = 2^(s - m_new) as the A fragments of the P V product, and the fp32 row
// sums over the quad.  P enters the product as two bf16 terms, hi = bf16(p)
// and lo = bf16(p - hi) (p - hi is exact in fp32), so the weights carry
// about 16 significant bits; the row sum uses the fp32 weights.
template <int BNK, bool LOWER8>
__device__ __forceinline__ void tile_probs(const float (&s)[BNK / 8][4], const float (&mnew)[2],
                                           uint32_t (&pa)[BNK / 16][4], uint32_t (&pl)[BNK / 16][4], float (&rs)[2]) {
  rs[0] = rs[1] = 0.f;
#pragma unroll
  for (int j = 0; j < BNK / 8; ++j) {
    float p[4], h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = e >> 1;
      if (LOWER8 && r == 1) {
        p[e] = h[e] = l[e] = 0.f;
        continue;
      }
      p[e] = (s[j][e] == -INFINITY) ? 0.f : ex2(__fsub_rn(s[j][e], mnew[r]));
      h[e] = bf16_round(p[e]);
      l[e] = __fsub_rn(p[e], h[e]);
    }
    rs[0] = __fadd_rn(__fadd_rn(rs[0], p[0]), p[1]);
    rs[1] = __fadd_rn(__fadd_rn(rs[1], p[2]), p[3]);
    pa[j >> 1][(j & 1) * 2 + 0] = pack_bf16x2(h[0], h[1]);
    pa[j >> 1][(j & 1) * 2 + 1] = pack_bf16x2(h[2], h[3]);
    pl[j >> 1][(j & 1) * 2 + 0] = pack_bf16x2(l[0], l[1]);
    pl[j >> 1][(j & 1) * 2 + 1] = pack_bf16x2(l[2], l[3]);
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    if (LOWER8 && r == 1) continue;
    rs[r] = __fadd_rn(rs[r], __shfl_xor_sync(0xffffffffu, rs[r], 1));
    rs[r] = __fadd_rn(rs[r], __shfl_xor_sync(0xffffffffu, rs[r], 2));
  }
}

// l <- l alpha + (the tile's row sum) for a row that saw a key of the tile.
__device__ __forceinline__ void tile_update_l(float& l, float alpha, float rs, bool rv) {
  l = rv ? __fadd_rn(__fmul_rn(l, alpha), rs) : l;
}

// O <- O alpha (with LOWER8 rows 8..15 have alpha 1 and are never stored).
template <int ND, bool LOWER8>
__device__ __forceinline__ void tile_rescale(float (&o)[ND / 8][4], const float (&alpha)[2]) {
#pragma unroll
  for (int n = 0; n < ND / 8; ++n) {
    o[n][0] = __fmul_rn(o[n][0], alpha[0]);
    o[n][1] = __fmul_rn(o[n][1], alpha[0]);
    if (!LOWER8) {
      o[n][2] = __fmul_rn(o[n][2], alpha[1]);
      o[n][3] = __fmul_rn(o[n][3], alpha[1]);
    }
  }
}

// O += P_hi V, P_lo V over the tile's two 16-key steps, for the output dims
// [dim0, dim0 + ND); per 8-dim block the order is hi, lo, hi, lo.  Each V
// fragment is loaded right before its products (the tile-at-a-time order).
template <int HD, int BNK, int ND>
__device__ __forceinline__ void tile_pv(float (&o)[ND / 8][4], const uint32_t (&pa)[BNK / 16][4],
                                        const uint32_t (&pl)[BNK / 16][4], uint32_t vbase, int lane, int dim0) {
  const int mi = lane >> 3, r8 = lane & 7;
  const int np0 = dim0 / 16;
#pragma unroll
  for (int ks = 0; ks < BNK / 16; ++ks) {
#pragma unroll
    for (int np = 0; np < ND / 16; ++np) {
      uint32_t b[4];
      ldmatrix_x4_trans(b, vbase + kv_off<HD>(ks * 16 + (mi & 1) * 8 + r8, (np0 + np) * 2 + (mi >> 1)));
      mma_bf16_16816(o[2 * np], pa[ks], b);
      mma_bf16_16816(o[2 * np], pl[ks], b);
      mma_bf16_16816(o[2 * np + 1], pa[ks], b + 2);
      mma_bf16_16816(o[2 * np + 1], pl[ks], b + 2);
    }
  }
}

// The same products in two steps, so that a tile's V fragments can be
// loaded while the previous tile's products run: the fragments for the
// output dims [dim0, dim0 + ND) per 16-key step and 16-dim block ...
template <int HD, int BNK, int ND>
__device__ __forceinline__ void tile_v_frags(uint32_t (&vb)[BNK / 16][ND / 16][4], uint32_t vbase, int lane,
                                             int dim0) {
  const int mi = lane >> 3, r8 = lane & 7;
  const int np0 = dim0 / 16;
#pragma unroll
  for (int ks = 0; ks < BNK / 16; ++ks)
#pragma unroll
    for (int np = 0; np < ND / 16; ++np)
      ldmatrix_x4_trans(vb[ks][np], vbase + kv_off<HD>(ks * 16 + (mi & 1) * 8 + r8, (np0 + np) * 2 + (mi >> 1)));
}

// ... then the products, in tile_pv's order.
template <int BNK, int ND>
__device__ __forceinline__ void tile_pv_mma(float (&o)[ND / 8][4], const uint32_t (&pa)[BNK / 16][4],
                                            const uint32_t (&pl)[BNK / 16][4],
                                            const uint32_t (&vb)[BNK / 16][ND / 16][4]) {
#pragma unroll
  for (int ks = 0; ks < BNK / 16; ++ks) {
#pragma unroll
    for (int np = 0; np < ND / 16; ++np) {
      mma_bf16_16816(o[2 * np], pa[ks], vb[ks][np]);
      mma_bf16_16816(o[2 * np], pl[ks], vb[ks][np]);
      mma_bf16_16816(o[2 * np + 1], pa[ks], vb[ks][np] + 2);
      mma_bf16_16816(o[2 * np + 1], pl[ks], vb[ks][np] + 2);
    }
  }
}

// One key tile for the 16 rows of a warp, which accumulates output dims
// [dim0, dim0 + ND).  S and the softmax state are computed over the full
// head either way, so every output element gets the same instruction chain
// whether one warp owns all dims or several warps share them.
template <int HD, int BNK, int ND, bool LOWER8>
__device__ __forceinline__ void attn_tile(RowState<ND>& st, const uint32_t (&qf)[HD / 16][4], uint32_t kbase,
                                          uint32_t vbase, int key0, const int (&pos)[2], const int (&lo)[2],
                                          float scale_log2, int lane, int dim0) {
  float s[BNK / 8][4], mx[2], mnew[2], alpha[2], rs[2];
  bool rv[2];
  uint32_t pa[BNK / 16][4], pl[BNK / 16][4];
  tile_scores<HD, BNK>(s, qf, kbase, lane);
  tile_mask_max<BNK, LOWER8>(s, mx, key0, pos, lo, scale_log2, lane);
#pragma unroll
  for (int r = 0; r < 2; ++r) tile_running_max(st.m[r], mx[r], mnew[r], alpha[r], rv[r]);
  tile_probs<BNK, LOWER8>(s, mnew, pa, pl, rs);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    tile_update_l(st.l[r], alpha[r], rs[r], rv[r]);
    st.m[r] = mnew[r];
  }
  tile_rescale<ND, LOWER8>(st.o, alpha);
  tile_pv<HD, BNK, ND>(st.o, pa, pl, vbase, lane, dim0);
}

}  // namespace vd
