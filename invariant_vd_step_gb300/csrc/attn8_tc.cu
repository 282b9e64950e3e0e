// Attention over the 8-bit KV cache for long row blocks: 5th-generation tensor
// cores (tcgen05), head dimensions 64 and 128.
//
// The rows, pages, chunks and splits, the arithmetic of a row and its order are
// those of attn8.cu (its header has the formulas), bit for bit: a tcgen05 K = 16
// step over fp16 operands gives what an mma.sync m16n8k16 step gives, and both
// kernels take the same steps (tests compare them).
//
// A CTA owns up to 256 rows of one (request, KV head), as two tiles of 128 (the
// MMA's M), and a range of splits, whose chunks of 128 keys it takes one after
// another.  Per chunk and tile: S = Q K^T (N = 128) into tensor memory; the
// tile's 128 softmax threads, one row each, take the chunk's maximum, turn S into
// fp16 weights in its place, and O = P V of the chunk goes to columns of its own,
// which the same threads fold into the split's O in their registers.  While one
// tile's softmax runs, the other tile's products do.  What it takes per chunk and
// SM: the products 2048 cycles at the dense rate, 32768 exponentials and about
// 1600 issue slots per scheduler in the softmax warps.
//
// Four warps turn the codes into the operands: a lane's operand words (kv8.cuh)
// are rows of 64 fp16 with the 128-byte swizzle after two 4-byte stores each, V
// transposed ([dim][key]) so that both operands are K-major.  The pages that are
// some row's own enter as a second K/V stage of their chunk, in bf16 scaled per
// token to exact fp16, with scores of their own; a row takes 16 of their columns.
//
// Roles (512 threads): warp 0 allocates tensor memory, its lane 0 issues the
// MMAs; warps 4..7 convert; warps 8..11 and 12..15 are the tiles' softmax.  Every
// wait is bounded.
#include <math.h>

#include "kv8.cuh"
#include "vd_internal.h"

namespace vd {
namespace {

constexpr int kSplit8 = 512, kChunk8 = 128, kChunkPages = 8;

template <int HD>
struct Tc8Cfg {
  static constexpr int ROWS = 128;
  static constexpr int Q_BYTES = ROWS * HD * 2;     // one tile: [hd block][row][64]
  static constexpr int K_BYTES = kChunk8 * HD * 2;  // [hd block][key][64]
  static constexpr int V_BYTES = kChunk8 * HD * 2;  // [key block][dim][64]
  static constexpr int STAGES = 2;
  static constexpr int SCALES = kChunk8 * 3 * 4;    // per stage: 8 pages or 128 tokens x (K scale, log2 of V's, 1 / V's)
  static constexpr int SC_RING = 4;
  static constexpr int SMEM = 1024 + 2 * Q_BYTES + STAGES * (K_BYTES + V_BYTES) + SC_RING * SCALES + 256;
  static constexpr int TMEM_COLS = 512;  // tile t: scores (then weights) from 128 t, O of a chunk from 256 + 128 t
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {  // fp16 A and B (K-major), fp32 D
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// 32 columns of this thread's lane; the values may be used after wait_ld32.
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void wait_ld32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t (&r)[16]) {  // waits
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Item: its request, rows [r0, r0 + n_rows) and splits [sp0, sp1).
template <int HD, int FMT>
__global__ void __launch_bounds__(512, 1) attn8_tc_kernel(Attn8Args a) {
  using C = Tc8Cfg<HD>;
  constexpr int KK = HD / 16, UNITS = Kv8Cfg<HD>::UNITS, PART = Kv8Cfg<HD>::PART;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sq = smem;
  uint8_t* sk = sq + 2 * C::Q_BYTES;               // K of stage s at sk + s * K_BYTES
  uint8_t* sv = sk + C::STAGES * C::K_BYTES;
  float* scales = reinterpret_cast<float*>(sv + C::STAGES * C::V_BYTES);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(scales) + C::SC_RING * C::SCALES);
  uint64_t* v_full = k_full + 2;
  uint64_t* k_empty = v_full + 2;
  uint64_t* v_empty = k_empty + 2;
  uint64_t* q_full = v_empty + 2;    // [tile] (and everything below)
  uint64_t* s_full = q_full + 2;     // scores of a chunk, and O of the chunk before, are there
  uint64_t* s16_full = s_full + 2;   // scores of the own pages
  uint64_t* o_free = s16_full + 2;   // O of the chunk before has been folded (chunks with own pages)
  uint64_t* p_full = o_free + 2;     // weights are there
  uint64_t* o_full = p_full + 2;     // O of the last chunk
  uint64_t* mma_done = o_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ int skip;
  const int kvh = blockIdx.x % a.Hkv;
  const int4 d0 = a.items[2 * (blockIdx.x / a.Hkv)], d1 = a.items[2 * (blockIdx.x / a.Hkv) + 1];
  const int b = d0.x, q0 = d0.y, qlen = d0.z, cached = d0.w, sp0 = d1.x, r0 = d1.y, sp1 = d1.z;
  const int G = a.Hq / a.Hkv, rows = qlen * G, kv_len = cached + qlen;
  const int r_end = min(rows, r0 + 256);
  const int ntile = r_end - r0 > 128 ? 2 : 1;
  const int p_min = cached + r0 / G, p_max = cached + (r_end - 1) / G;
  const int lo_min = a.window > 0 ? max(0, p_min - a.window + 1) : 0;
  const int own_lo = p_min >> 4, own_hi = p_max >> 4;
  const int ch0 = max(sp0 * (kSplit8 / kChunk8), lo_min / kChunk8);
  const int ch1 = min(sp1 * (kSplit8 / kChunk8) - 1, p_max / kChunk8);  // last chunk
  if (threadIdx.x == 0) {
    skip = a.status ? *reinterpret_cast<volatile int*>(a.status) : 0;
    for (int k = 0; k < 2; ++k) {
      mbar_init(&k_full[k], 128);
      mbar_init(&v_full[k], 128);
      mbar_init(&k_empty[k], 1);
      mbar_init(&v_empty[k], 1);
      mbar_init(&q_full[k], 128);
      mbar_init(&s_full[k], 1);
      mbar_init(&s16_full[k], 1);
      mbar_init(&o_free[k], 128);
      mbar_init(&p_full[k], 128);
      mbar_init(&o_full[k], 1);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  if (skip || ch0 > ch1) return;  // nothing to see here
  if (warp == 0) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto diag = [&](int ch) { return own_lo <= ch * kChunkPages + kChunkPages - 1 && own_hi >= ch * kChunkPages; };
  // pages of chunk ch that some row sees in 8 bits, and those that are some row's own (numbers within the chunk)
  auto lo8 = [&](int ch) { return max(0, (lo_min >> 4) - ch * kChunkPages); };
  auto hi8 = [&](int ch) { return min(kChunkPages, own_hi - ch * kChunkPages); };
  auto lo16 = [&](int ch) { return max(0, own_lo - ch * kChunkPages); };
  auto hi16 = [&](int ch) { return min(kChunkPages, own_hi + 1 - ch * kChunkPages); };

  if (warp < 4) {
    regs_dec<40>();
    if (warp == 0 && lane == 0) {
      const uint32_t id_s = idesc_f16(128, kChunk8), id_pv = idesc_f16(128, HD);
      const uint32_t q_lo = sw128_desc_lo(smem_u32(sq)), k_lo = sw128_desc_lo(smem_u32(sk)), v_lo = sw128_desc_lo(smem_u32(sv));
      auto wait = [&](uint64_t* f, int n) { return mbar_wait(f, n & 1, abort_flag, a.status); };
      // scores of tile t against the K of stage st into columns `col`
      auto scores = [&](int t, int st, uint32_t col) {
        const uint32_t q = q_lo + t * (C::Q_BYTES >> 4), k = k_lo + (st & 1) * (C::K_BYTES >> 4);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
          umma_bf16_lo(tmem + col, q + (kk >> 2) * (C::ROWS * 128 >> 4) + 2 * (kk & 3),
                       k + (kk >> 2) * (kChunk8 * 128 >> 4) + 2 * (kk & 3), id_s, kk ? 1u : 0u);
      };
      // O of tile t += weights of pages [x0, x1) in columns `p` times the V of stage st; first: from zero
      auto pv = [&](int t, int st, uint32_t p, int x0, int x1, bool first) {
        const uint32_t v = v_lo + (st & 1) * (C::V_BYTES >> 4);
        for (int x = x0; x < x1; ++x)
          umma_bf16_ta(tmem + 256 + 128 * t, tmem + p + 8 * x, v + (x >> 2) * (HD * 128 >> 4) + 2 * (x & 3), id_pv,
                       first && x == x0 ? 0u : 1u);
      };
      int n16[2] = {0, 0};
      bool ok = true;
      for (int t = 0; t < ntile; ++t) ok = ok && wait(&q_full[t], 0);
      // P V of chunk ch, whose stages are st (and st + 1), number it
      auto chunk_pv = [&](int t, int ch, int st, int it) {
        if (!wait(&p_full[t], it) || !wait(&v_full[st & 1], st >> 1)) return false;
        const bool dg = diag(ch);
        if (dg && !wait(&v_full[(st + 1) & 1], (st + 1) >> 1)) return false;
        tc_fence_after();
        pv(t, st, 128 * t, lo8(ch), hi8(ch), true);
        if (dg) pv(t, st + 1, 128 * t + 64, lo16(ch), hi16(ch), lo8(ch) >= hi8(ch));
        return true;
      };
      int st = 0, st_prev = 0;
      for (int ch = ch0; ok && ch <= ch1; ++ch) {
        const int it = ch - ch0;
        ok = wait(&k_full[st & 1], st >> 1);
        for (int t = 0; ok && t < ntile; ++t) {
          if (it > 0) ok = chunk_pv(t, ch - 1, st_prev, it - 1);
          if (!ok) break;
          tc_fence_after();
          scores(t, st, 128 * t);
          umma_commit(&s_full[t]);
        }
        if (!ok) break;
        umma_commit(&k_empty[st & 1]);
        if (it > 0) {
          umma_commit(&v_empty[st_prev & 1]);
          if (diag(ch - 1)) umma_commit(&v_empty[(st_prev + 1) & 1]);
        }
        st_prev = st++;
        if (diag(ch)) {
          ok = wait(&k_full[st & 1], st >> 1);
          for (int t = 0; ok && t < ntile; ++t) {
            ok = wait(&o_free[t], n16[t]++);
            if (!ok) break;
            tc_fence_after();
            scores(t, st, 256 + 128 * t);
            umma_commit(&s16_full[t]);
          }
          if (!ok) break;
          umma_commit(&k_empty[st & 1]);
          ++st;
        }
      }
      for (int t = 0; ok && t < ntile; ++t) {
        ok = chunk_pv(t, ch1, st_prev, ch1 - ch0);
        if (ok) umma_commit(&o_full[t]);
      }
      umma_commit(mma_done);
    }
  } else if (warp < 8) {
    // ---- operands.  Each warp takes two pages of a stage's K, then of its V.
    regs_dec<88>();
    const int cw = warp - 4, g = lane >> 2, t4 = lane & 3;
    uint4 w[2][UNITS];
    const int* pt = a.page_table + static_cast<size_t>(b) * a.pt_stride;
    int st = 0;
    bool ok = true;
    auto warp_wait = [&](uint64_t* f, int n) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(f, n & 1, abort_flag, a.status));
      return ok;
    };
    auto load = [&](int ch, bool v, const int (&pid)[2]) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint4* src = reinterpret_cast<const uint4*>(a.codes + (static_cast<size_t>(pid[x]) * a.Hkv + kvh) * (2 * PART) + (v ? PART : 0));
        const bool in = 2 * cw + x >= lo8(ch) && 2 * cw + x < hi8(ch);
#pragma unroll
        for (int u = 0; u < UNITS; ++u) w[x][u] = in ? __ldcg(src + u * 32 + lane) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    auto ids = [&](int ch, int (&pid)[2]) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int pg = 2 * cw + x;
        pid[x] = ch <= ch1 && pg >= lo8(ch) && pg < hi8(ch) ? pt[ch * kChunkPages + pg] : 0;
      }
    };
    // One operand word: two fp16 pairs of row `row` (row % 8 = g), at 16-byte columns c and c + 1.
    auto put = [&](uint32_t base, int row, int c, uint32_t word) {
      uint32_t lo, hi;
      kv8_expand<FMT>(word, lo, hi);
      const uint32_t at = base + row * 128 + t4 * 4;
      sts32(at + ((c ^ g) << 4), lo);
      sts32(at + (((c + 1) ^ g) << 4), hi);
    };
    int pid[2], pid_next[2];
    ids(ch0, pid);
    load(ch0, false, pid);
    for (int ch = ch0; ok && ch <= ch1; ++ch) {
      ids(ch + 1, pid_next);
      if (st >= 2 && !warp_wait(&k_empty[st & 1], (st >> 1) - 1)) break;
      float* sc = scales + (st & 3) * (C::SCALES / 4);
      if (lane < 2) {
        const int x = 2 * cw + lane;
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (x >= lo8(ch) && x < hi8(ch)) f = __ldcg(a.scales + static_cast<size_t>(lane ? pid[1] : pid[0]) * a.Hkv + kvh);
        sc[x * 4] = f.x;
        sc[x * 4 + 1] = f.z;
        sc[x * 4 + 2] = f.y;
      }
      {
        const uint32_t base = smem_u32(sk + (st & 1) * C::K_BYTES);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int row = (2 * cw + x) * 16 + g;
#pragma unroll
          for (int u = 0; u < UNITS; ++u) {  // k-steps 2 u and 2 u + 1; key blocks 0 and 1
            const uint32_t blk = base + (u >> 1) * (kChunk8 * 128);
            const int c = (u & 1) * 4;
            put(blk, row, c, w[x][u].x);
            put(blk, row + 8, c, w[x][u].y);
            put(blk, row, c + 2, w[x][u].z);
            put(blk, row + 8, c + 2, w[x][u].w);
          }
        }
      }
      load(ch, true, pid);
      fence_proxy_async_smem();
      mbar_arrive(&k_full[st & 1]);
      if (st >= 2 && !warp_wait(&v_empty[st & 1], (st >> 1) - 1)) break;
      {
        const uint32_t base = smem_u32(sv + (st & 1) * C::V_BYTES);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int page = 2 * cw + x;
          const uint32_t blk = base + (page >> 2) * (HD * 128);
          const int c = (page & 3) * 2;
#pragma unroll
          for (int u = 0; u < UNITS; ++u) {
            put(blk, 32 * u + g, c, w[x][u].x);
            put(blk, 32 * u + 8 + g, c, w[x][u].y);
            put(blk, 32 * u + 16 + g, c, w[x][u].z);
            put(blk, 32 * u + 24 + g, c, w[x][u].w);
          }
        }
      }
      pid[0] = pid_next[0];
      pid[1] = pid_next[1];
      if (ch < ch1) load(ch + 1, false, pid);
      fence_proxy_async_smem();
      mbar_arrive(&v_full[st & 1]);
      ++st;
      if (diag(ch)) {
        // the own pages in bf16: lane (token, half of the head dimension); the scales of a token that is not finite
        // are NaN, and its V counts as 0 (its weight is NaN, or 0 where it is not seen)
        if (st >= 2 && !(warp_wait(&k_empty[st & 1], (st >> 1) - 1) && warp_wait(&v_empty[st & 1], (st >> 1) - 1))) break;
        float* so = scales + (st & 3) * (C::SCALES / 4);
        const int token = lane >> 1, half = lane & 1;
        for (int x = 0; x < 2; ++x) {
          const int pg = 2 * cw + x, page = ch * kChunkPages + pg;
          if (pg < lo16(ch) || pg >= hi16(ch)) continue;
          const int phys = a.open_table[static_cast<size_t>(b) * a.open_stride + page - (cached >> 4)];
          const bool have = page * 16 + token < kv_len;
          const int key = pg * 16 + token;
          for (int v = 0; v < 2; ++v) {
            const uint4* src = reinterpret_cast<const uint4*>(a.open + ((static_cast<size_t>(phys) * 2 + v) * a.Hkv + kvh) * PART +
                                                              token * HD + half * (HD / 2));
            uint32_t mx = 0u;
#pragma unroll
            for (int i = 0; i < HD / 16; ++i) {
              const uint4 y = have ? __ldcg(src + i) : make_uint4(0u, 0u, 0u, 0u);
              mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(y.x & 0x7fff7fffu, y.y & 0x7fff7fffu),
                                         __vmaxu2(y.z & 0x7fff7fffu, y.w & 0x7fff7fffu)));
            }
            mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            const int e = kv8_exp(kv8_max_halves(mx));
            const float up = kv8_up(e);
            if (half == 0) {
              if (v == 0) {
                so[key] = e == 255 ? kv8_nan() : kv8_down(e);
              } else {
                so[kChunk8 + key] = e == 255 ? kv8_nan() : kv8_log2_down(e);
                so[2 * kChunk8 + key] = up;
              }
            }
#pragma unroll 2
            for (int i = 0; i < HD / 16; ++i) {
              uint4 y = have ? __ldcg(src + i) : make_uint4(0u, 0u, 0u, 0u);
              y = make_uint4(kv8_to_f16(y.x, up), kv8_to_f16(y.y, up), kv8_to_f16(y.z, up), kv8_to_f16(y.w, up));
              const int d = half * (HD / 2) + i * 8;  // dims d .. d + 7
              if (v == 0) {
                *reinterpret_cast<uint4*>(sk + (st & 1) * C::K_BYTES + (d >> 6) * (kChunk8 * 128) + key * 128 +
                                          ((((d >> 3) & 7) ^ (key & 7)) << 4)) = y;
              } else {
                if (e == 255) y = make_uint4(0u, 0u, 0u, 0u);
                uint8_t* to = sv + (st & 1) * C::V_BYTES + (key >> 6) * (HD * 128) + (key & 7) * 2;
                const uint32_t h[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  *reinterpret_cast<uint16_t*>(to + (d + k) * 128 + ((((key >> 3) & 7) ^ ((d + k) & 7)) << 4)) =
                      static_cast<uint16_t>(h[k >> 1] >> (16 * (k & 1)));
              }
            }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&k_full[st & 1]);
        mbar_arrive(&v_full[st & 1]);
        ++st;
      }
    }
  } else {
    // ---- softmax: one row per thread
    regs_inc<192>();
    const int t = (warp - 8) >> 2, lr = (warp & 3) * 32 + lane, row = r0 + t * 128 + lr;
    const bool valid = row < r_end;
    const int tok = valid ? row / G : 0, hq = kvh * G + (valid ? row % G : 0);
    const int pos = valid ? cached + tok : -1, own = pos >> 4;
    const int lo = valid ? (a.window > 0 ? max(0, pos - a.window + 1) : 0) : 1;
    if (t < ntile) {
      float rowfac;
      {  // the row's query -> [hd block][row][64] fp16, 128-byte swizzle
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (static_cast<size_t>(q0 + tok) * a.Hq + hq) * HD);
        uint4 x[HD / 8];
        uint32_t mx = 0u;
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) x[i] = valid ? src[i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < HD / 8; ++i)
          mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                     __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
        const int e = kv8_exp(kv8_max_halves(mx));
        const float up = kv8_up(e);
        rowfac = e == 255 ? kv8_nan() : __fmul_rn(a.scale_log2, kv8_down(e));
#pragma unroll
        for (int i = 0; i < HD / 8; ++i)
          *reinterpret_cast<uint4*>(sq + t * C::Q_BYTES + (i >> 3) * (C::ROWS * 128) + lr * 128 + (((i & 7) ^ (lr & 7)) << 4)) =
              make_uint4(kv8_to_f16(x[i].x, up), kv8_to_f16(x[i].y, up), kv8_to_f16(x[i].z, up), kv8_to_f16(x[i].w, up));
        fence_proxy_async_smem();
        mbar_arrive(&q_full[t]);
      }
      const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      const uint32_t s_at = lanes + 128 * t, o_at = lanes + 256 + 128 * t;
      bool ok = true;
      auto warp_wait = [&](uint64_t* f, int n) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(f, n & 1, abort_flag, a.status));
        return ok;
      };
      float M = 0.f, L = 0.f, O[HD];
      bool any = false;          // O holds chunks of the split in hand
      float mc = 0.f, lc = 0.f;  // of the chunk whose O is still in tensor memory
      // Folds that chunk (number ch) into the split's state, and stores the split's if it was its last
      auto fold = [&](int ch) {
        const bool sees = valid && max(lo, ch * kChunk8) <= min(pos, ch * kChunk8 + kChunk8 - 1);
        const float mn = any ? fmaxf(M, mc) : mc;
        const float ca = ex2(__fsub_rn(M, mn)), cb = ex2(__fsub_rn(mc, mn));
#pragma unroll
        for (int c = 0; c < HD / 32; ++c) {
          uint32_t x[32];
          ld32(o_at + 32 * c, x);
          wait_ld32(x);
          if (sees) {
            if (any) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                O[32 * c + i] = __fadd_rn(__fmul_rn(O[32 * c + i], ca), __fmul_rn(__uint_as_float(x[i]), cb));
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) O[32 * c + i] = __uint_as_float(x[i]);
            }
          }
        }
        if (sees) {
          L = any ? __fadd_rn(__fmul_rn(L, ca), __fmul_rn(lc, cb)) : lc;
          M = mn;
          any = true;
        }
        if ((ch & 3) == 3 || ch == ch1) {
          if (any) {
            const size_t base = (static_cast<size_t>(q0 + tok) * a.Hq + hq) * a.max_splits + (ch >> 2);
            a.part_ml[base * 2] = M;
            a.part_ml[base * 2 + 1] = L;
            float4* po = reinterpret_cast<float4*>(a.part_o + base * HD);
#pragma unroll
            for (int i = 0; i < HD / 4; ++i) po[i] = make_float4(O[4 * i], O[4 * i + 1], O[4 * i + 2], O[4 * i + 3]);
          }
          any = false;
        }
      };
      int st = 0, n16 = 0;
      for (int ch = ch0; ch <= ch1; ++ch) {
        const int it = ch - ch0, pg0 = ch * kChunkPages;
        if (!warp_wait(&s_full[t], it)) break;
        tc_fence_after();
        if (it > 0) fold(ch - 1);
        const float* sc = scales + (st & 3) * (C::SCALES / 4);
        const bool dg = diag(ch);
        const float* so = scales + ((st + 1) & 3) * (C::SCALES / 4);
        if (dg) {
          tc_fence_before();
          mbar_arrive(&o_free[t]);
          if (!warp_wait(&s16_full[t], n16++)) break;
          tc_fence_after();
        }
        st += dg ? 2 : 1;
        // every row of the warp sees the whole chunk in 8 bits (rows that are none aside)
        const bool full = __all_sync(0xffffffffu, !valid || (lo <= ch * kChunk8 && own >= pg0 + kChunkPages));
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t x[32];
          ld32(s_at + 32 * c, x);
          wait_ld32(x);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int pg = 2 * c + h;
            const float ks = __fmul_rn(sc[pg * 4], rowfac), lv = sc[pg * 4 + 1];
            if (full) {
#pragma unroll
              for (int i = 0; i < 16; ++i) mx = fmaxf(mx, __fmaf_rn(__uint_as_float(x[16 * h + i]), ks, lv));
            } else if (pg0 + pg < own) {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if ((pg0 + pg) * 16 + i >= lo) mx = fmaxf(mx, __fmaf_rn(__uint_as_float(x[16 * h + i]), ks, lv));
            }
          }
        }
        const int x0 = lo16(ch), x1 = hi16(ch);
        if (dg) {
          for (int pg = x0; pg < x1; ++pg) {
            if (!__any_sync(0xffffffffu, own == pg0 + pg)) continue;
            uint32_t x[16];
            ld16(o_at + 16 * pg, x);
            if (own == pg0 + pg) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int key = (pg0 + pg) * 16 + i;
                const float v = __fmaf_rn(__uint_as_float(x[i]), __fmul_rn(so[pg * 16 + i], rowfac), so[kChunk8 + pg * 16 + i]);
                if (key >= lo && key <= pos) mx = fmaxf(mx, v);
              }
            }
          }
        }
        mc = mx;
        float l[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t x[32];
          ld32(s_at + 32 * c, x);
          wait_ld32(x);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int pg = 2 * c + h;
            const float ks = __fmul_rn(sc[pg * 4], rowfac), lv = sc[pg * 4 + 1], iv = sc[pg * 4 + 2];
            const bool mine = full || pg0 + pg < own;
            float p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float v = __fmaf_rn(__uint_as_float(x[16 * h + i]), ks, lv);
              if (!full && !(mine && (pg0 + pg) * 16 + i >= lo)) v = -INFINITY;
              p[i] = ex2(__fsub_rn(v, mx));
            }
            if (full || (mine && (pg0 + pg) * 16 + 15 >= lo)) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                l[k] = __fmaf_rn(__fadd_rn(__fadd_rn(p[2 * k], p[2 * k + 1]), __fadd_rn(p[2 * k + 8], p[2 * k + 9])), iv, l[k]);
            }
            uint32_t pk[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) pk[i] = pack_f16x2(p[2 * i], p[2 * i + 1]);
            st8(s_at + 8 * pg, pk);
          }
        }
        if (dg) {
          for (int pg = x0; pg < x1; ++pg) {
            uint32_t x[16], pk[8];
            ld16(o_at + 16 * pg, x);
            const bool mine = own == pg0 + pg;
            float p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int key = (pg0 + pg) * 16 + i;
              const float v = __fmaf_rn(__uint_as_float(x[i]), __fmul_rn(so[pg * 16 + i], rowfac), so[kChunk8 + pg * 16 + i]);
              p[i] = mine && key >= lo && key <= pos ? ex2(__fsub_rn(v, mx)) : 0.f;
            }
            if (mine) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float* up = so + 2 * kChunk8 + pg * 16 + 2 * k;
                l[k] = __fmaf_rn(p[2 * k], up[0], l[k]);
                l[k] = __fmaf_rn(p[2 * k + 1], up[1], l[k]);
                l[k] = __fmaf_rn(p[2 * k + 8], up[8], l[k]);
                l[k] = __fmaf_rn(p[2 * k + 9], up[9], l[k]);
              }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) pk[i] = pack_f16x2(p[2 * i], p[2 * i + 1]);
            st8(s_at + 64 + 8 * pg, pk);
          }
        }
        lc = __fadd_rn(__fadd_rn(l[0], l[1]), __fadd_rn(l[2], l[3]));
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[t]);
      }
      if (ok && warp_wait(&o_full[t], 0)) {
        tc_fence_after();
        fold(ch1);
      }
    }
  }
  // Teardown: issued MMAs finish, then tensor memory is freed.
  if (warp == 0 && lane == 0) drain_wait(mma_done, 0);
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int HD, int FMT>
int launch_attn8_tc_t(const Attn8Args& a, int n_blocks, cudaStream_t s) {
  using C = Tc8Cfg<HD>;
  VD_CUDA_TRY(cudaFuncSetAttribute(attn8_tc_kernel<HD, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM));
  VD_CUDA_TRY(launch_k(attn8_tc_kernel<HD, FMT>, dim3(static_cast<unsigned>(n_blocks) * a.Hkv), dim3(512), C::SMEM, s, a));
  return VD_OK;
}

}  // namespace

int launch_attention8_tc(const Attn8Args& a, int hd, int format, int n_blocks, cudaStream_t s) {
  if (n_blocks <= 0) return VD_OK;
  if (hd == 64)
    return format == VD_KV8_INT8 ? launch_attn8_tc_t<64, kKv8Int8>(a, n_blocks, s) : launch_attn8_tc_t<64, kKv8E4m3>(a, n_blocks, s);
  if (hd == 128)
    return format == VD_KV8_INT8 ? launch_attn8_tc_t<128, kKv8Int8>(a, n_blocks, s) : launch_attn8_tc_t<128, kKv8E4m3>(a, n_blocks, s);
  return fail(VD_ERR_UNSUPPORTED, "the tcgen05 kernel of the 8-bit cache takes head_dim 64 or 128");
}

}  // namespace vd
