// Attention over the 8-bit KV cache for long row blocks: 5th-generation tensor
// cores (tcgen05).
//
// The rows, pages, chunks and splits, the arithmetic of a row and its order are
// those of attn8.cu (its header has the formulas), bit for bit: a tcgen05 K = 16
// step over fp16 operands gives what an mma.sync m16n8k16 step gives, and both
// kernels take the same steps (tests compare them).
//
// A CTA owns up to 128 rows (the MMA's M) of one (request, KV head) and a run of
// splits, whose chunks of 128 keys it takes one after another.  Per chunk: S = Q
// K^T (N = 128) into one of two score buffers of tensor memory; the softmax
// threads, two per row with 64 keys each, take the row's maximum, turn S into
// fp16 weights in its place, and fold O = P V of the chunk before (half of the dims
// each) into the split's O in their registers; P V and the scores of the chunk
// after the next run meanwhile.  A run that holds all of a block's splits folds
// them too, as the merge kernel does (its totals wait in tensor memory while a
// split is in hand), and writes the output; shorter runs, which the last blocks of a
// launch are cut into, leave the splits' partials to that kernel.
//
// What a chunk takes per SM: the products 1024 cycles at the dense rate, 16384
// exponentials 512, 64 KB of operands from L2; about 1500 issue slots per
// scheduler, whose two softmax warps leave more than half of its cycles idle: that
// is what bounds it (3000 cycles per chunk).  Measured, 2048 tokens behind 6144
// keys, 32 heads over 8 of 128: 385 us, 625 TFLOP/s.  With one maximum for scores and V
// scales together, which loses weights, 371; before that 424 with the totals in
// global memory, two O buffers and one barrier of all softmax threads (the two of a
// row need only each other), 447 with the folding in four warps of its own, which
// became what the others waited for, and 414 with 216 registers in place of 232 (8 bytes
// of a thread still spill at head dimension 128, 108 at 256).
//
// Head dimension 256: a row block is two CTAs, each with all of the scores and half
// of the dims of V and O, so that tensor memory and registers hold what they hold at
// 128; K comes in two units of 128 dims.  512 tokens behind 4000, 8 heads over 4: 94 us
// where mma.sync takes 204.  (One unit of 256 dims, without a second one in flight:
// the same.)
//
// The operands are made once per launch, not once per row block: an expanding
// kernel turns every chunk of the launch's requests into an image of the two
// shared-memory tiles, rows of 64 fp16 with the 128-byte swizzle, V transposed
// ([dim][key]) so that both are K-major, and of the chunk's scales; a block then
// fetches a tile with one bulk copy (from L2: a request's blocks run together).
// The pages that are some row's own have a second image of their chunk, in bf16
// scaled per token to exact fp16, and scores of their own (in the other score
// buffer); a row takes 16 of their columns.  Converting inside the blocks, by eight
// warps beside the softmax, took a third of the issue slots: 738 us where the images
// came to 489.
//
// Roles (384 threads): warp 0 allocates tensor memory, its lane 0 issues the MMAs;
// warp 1's lane 0 the copies; warps 4..11 are the softmax.  Every wait is bounded.
#include <math.h>

#include "kv8.cuh"
#include "vd_internal.h"

namespace vd {
namespace {

constexpr int kSplit8 = 512, kChunk8 = 128, kChunkPages = 8;

template <int HD>
struct Tc8Cfg {
  static constexpr int ROWS = 128;
  static constexpr int Q_BYTES = ROWS * HD * 2;     // [hd block][row][64]
  static constexpr int K_BYTES = kChunk8 * HD * 2;  // [hd block][key][64]
  static constexpr int VD = HD < 128 ? HD : 128;    // dims of a block's O
  static constexpr int HALVES = HD / VD;            // blocks that share a row block's scores, each with VD of the dims
  static constexpr int V_BYTES = kChunk8 * VD * 2;  // [key block][dim][64]
  static constexpr int KU = HALVES;                 // units that K is copied in: of at most 128 dims
  static constexpr int KU_BYTES = K_BYTES / KU;
  static constexpr int STAGES = 2;                  // of K's units, and of V
  static constexpr int SCALES = kChunk8 * 2 * 4;    // per stage: 8 pages or 128 tokens x (K scale, log2 of V's)
  static constexpr int SC_RING = 4;
  static constexpr int NT = kChunkParts;  // softmax threads per row
  static constexpr int NS = 128 * NT;
  static constexpr int OUT_DIMS = HD <= 128 ? 32 : 16;
  static constexpr int OUT_BYTES = 4 * NT * 32 * OUT_DIMS * 4;  // per softmax warp: 32 rows x OUT_DIMS of float32
  static constexpr int SMEM = 1024 + Q_BYTES + STAGES * (KU_BYTES + V_BYTES) + OUT_BYTES + SC_RING * SCALES + 256;
  static constexpr int TMEM_COLS = 512;  // chunk c: scores (then weights) from 128 (c % 2), O from 256; the totals from 384
  static constexpr int THREADS = 128 + NS;
  // A chunk's image: K tile, V tiles, scales
  static constexpr int IMAGE = K_BYTES + HALVES * V_BYTES + SCALES;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {  // fp16 A and B (K-major), fp32 D
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Columns of this thread's lane; the values may be used after the wait_ld.
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, "
      "%23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void wait_ld32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
        "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
        "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
        "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]),
        "+r"(r[31])::"memory");
}
__device__ __forceinline__ void wait_ld16(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
        "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
        "+r"(r[15])::"memory");
}
__device__ __forceinline__ void st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
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

// Packed float32 pairs; each half rounded as the scalar operation rounds it.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t f2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ float f2_lo(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float f2_hi(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ uint64_t f2_fma(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t f2_sub(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}

// Barrier id of THREADS softmax threads that also tells whether any of them has
// given up.  The two threads of a row are in warps that share nothing with others,
// so these meet in barriers of their own.
template <int THREADS>
__device__ __forceinline__ bool softmax_sync(int id, bool ok) {
  uint32_t bad;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, %2, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(bad)
      : "r"(ok ? 0u : 1u), "r"(id), "n"(THREADS)
      : "memory");
  return bad == 0;
}

// Images of chunks: one block per (chunk, KV head, K or V), a warp per page.  A lane's
// operand words (kv8.cuh) become two 4-byte pieces of rows of the tiles, which
// leave shared memory in whole 16-byte words.  Bound by the latency of its pages: 16
// KB of codes in and 32 KB of fp16 out per block at hd 128, 512 such blocks a request
// of 4096 keys and 8 KV heads.
template <int HD, int FMT>
__global__ void __launch_bounds__(256, HD <= 128 ? 5 : 3) attn8_expand_kernel(Attn8Args a) {
  using C = Tc8Cfg<HD>;
  constexpr int UNITS = Kv8Cfg<HD>::UNITS, PART = Kv8Cfg<HD>::PART;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int pg = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int v = blockIdx.x & 1, block_of = blockIdx.x >> 1;  // K or V
  const int kvh = block_of % a.Hkv;
  const int4 d = a.chunks[2 * (block_of / a.Hkv)], e = a.chunks[2 * (block_of / a.Hkv) + 1];
  const int b = d.x, ch = d.y, image = d.z, cached = e.x, kv_len = e.y;
  const bool own = d.w != 0;  // the image of the chunk's own pages
  const int page = ch * kChunkPages + pg;
  const bool in = own ? page >= cached >> 4 && page * 16 < kv_len : (page + 1) * 16 <= kv_len;
  const int pid = !in ? 0
                  : own ? a.open_table[static_cast<size_t>(b) * a.open_stride + page - (cached >> 4)]
                        : a.page_table[static_cast<size_t>(b) * a.pt_stride + page];
  pdl_wait();
  pdl_trigger();
  static_assert(C::K_BYTES == C::HALVES * C::V_BYTES, "K's tile or V's");
  float* sc = reinterpret_cast<float*>(smem + C::K_BYTES);
  if (!own) {
    const size_t block = static_cast<size_t>(pid) * a.Hkv + kvh;
    const uint4* src = reinterpret_cast<const uint4*>(a.codes + block * (2 * PART)) + lane;
    uint4 w[UNITS];
#pragma unroll
    for (int u = 0; u < UNITS; ++u) w[u] = in ? __ldcg(src + v * (PART / 16) + u * 32) : make_uint4(0u, 0u, 0u, 0u);
    if (v == 0 && lane == 0) {
      const float4 f = in ? __ldcg(a.scales + block) : make_float4(0.f, 0.f, 0.f, 0.f);
      *reinterpret_cast<float2*>(sc + pg * 2) = make_float2(f.x, f.z);
    }
    // the two fp16 pairs of a word go to 16-byte columns c and c + 1 of row g of an 8-row group
    auto col = [&](int c) { return static_cast<uint32_t>(g * 128 + ((c ^ g) << 4) + t4 * 4); };
    auto put = [&](uint32_t at0, uint32_t at1, uint32_t word) {
      uint32_t lo, hi;
      kv8_expand<FMT>(word, lo, hi);
      sts32(at0, lo);
      sts32(at1, hi);
    };
    if (v == 0) {
      const uint32_t kb = smem_u32(smem) + pg * (16 * 128);
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {  // k-steps 2 u and 2 u + 1 of key blocks 0 and 1
        const int k = (u & 1) * 4, at = (u >> 1) * (kChunk8 * 128);
        put(kb + at + col(k), kb + at + col(k + 1), w[u].x);
        put(kb + at + 8 * 128 + col(k), kb + at + 8 * 128 + col(k + 1), w[u].y);
        put(kb + at + col(k + 2), kb + at + col(k + 3), w[u].z);
        put(kb + at + 8 * 128 + col(k + 2), kb + at + 8 * 128 + col(k + 3), w[u].w);
      }
    } else {
      // this page's 16 keys are columns 2 (page % 4) and + 1 of its key block
      const uint32_t vb = smem_u32(smem) + (pg >> 2) * (C::VD * 128), c0 = vb + col((pg & 3) * 2), c1 = vb + col((pg & 3) * 2 + 1);
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {  // dims 32 u .. + 31
        const int at = 32 * u / C::VD * C::V_BYTES + 32 * u % C::VD * 128;
        put(c0 + at, c1 + at, w[u].x);
        put(c0 + at + 8 * 128, c1 + at + 8 * 128, w[u].y);
        put(c0 + at + 16 * 128, c1 + at + 16 * 128, w[u].z);
        put(c0 + at + 24 * 128, c1 + at + 24 * 128, w[u].w);
      }
    }
  } else {
    // The own pages in bf16, eight tokens at a time, four lanes a token; zeros behind
    // the last token and in other pages.  The scales of a token that is not finite are
    // NaN, and its V counts as 0 (its weight is NaN, or 0 where it is not seen).
    const __nv_bfloat16* src = a.open + ((static_cast<size_t>(pid) * 2 + v) * a.Hkv + kvh) * PART + t4 * (HD / 4);
#pragma unroll
    for (int token = g; token < 16; token += 8) {
      const int key = pg * 16 + token;
      const bool have = in && page * 16 + token < kv_len;
      uint4 y[HD / 32];
      uint32_t mx = 0u;
#pragma unroll
      for (int i = 0; i < HD / 32; ++i)
        y[i] = have ? __ldcg(reinterpret_cast<const uint4*>(src + token * HD) + i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int i = 0; i < HD / 32; ++i)
        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(y[i].x & 0x7fff7fffu, y[i].y & 0x7fff7fffu),
                                   __vmaxu2(y[i].z & 0x7fff7fffu, y[i].w & 0x7fff7fffu)));
      mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int ex = kv8_exp(kv8_max_halves(mx));
      const float up = kv8_up(ex);
      if (t4 == 0) {
        if (v == 0) {
          sc[key] = ex == 255 ? kv8_nan() : kv8_down(ex);
        } else {
          sc[kChunk8 + key] = ex == 255 ? kv8_nan() : kv8_log2_down(ex);
        }
      }
#pragma unroll
      for (int i = 0; i < HD / 32; ++i) {
        const uint32_t x[4] = {kv8_to_f16(y[i].x, up), kv8_to_f16(y[i].y, up), kv8_to_f16(y[i].z, up), kv8_to_f16(y[i].w, up)};
        const int dim = t4 * (HD / 4) + i * 8;  // .. + 7
        if (v == 0) {
          *reinterpret_cast<uint4*>(smem + (dim >> 6) * (kChunk8 * 128) + key * 128 + ((((dim >> 3) & 7) ^ (key & 7)) << 4)) =
              make_uint4(x[0], x[1], x[2], x[3]);
        } else {
          uint8_t* to = smem + dim / C::VD * C::V_BYTES + (key >> 6) * (C::VD * 128) + (key & 7) * 2 + dim % C::VD * 128;
#pragma unroll
          for (int k = 0; k < 8; ++k)  // (dim % 8 = 0)
            *reinterpret_cast<uint16_t*>(to + k * 128 + ((((key >> 3) & 7) ^ k) << 4)) =
                ex == 255 ? static_cast<uint16_t>(0) : static_cast<uint16_t>(x[k >> 1] >> (16 * (k & 1)));
        }
      }
    }
  }
  __syncthreads();
  uint8_t* image_at = a.images + (static_cast<size_t>(image) * a.Hkv + kvh) * C::IMAGE;
  uint4* to = reinterpret_cast<uint4*>(image_at + v * C::K_BYTES);
  const uint4* from = reinterpret_cast<const uint4*>(smem);
#pragma unroll 4
  for (int i = threadIdx.x; i < C::K_BYTES / 16; i += 256) to[i] = from[i];
  // scales: of an 8-bit chunk's pages, by K's block; of own tokens K's, then V's
  const int s0 = own && v ? kChunk8 / 4 : 0, s1 = !own ? (v ? 0 : kChunkPages / 2) : v ? C::SCALES / 16 : kChunk8 / 4;
  to = reinterpret_cast<uint4*>(image_at + 2 * C::K_BYTES);
  for (int i = s0 + threadIdx.x; i < s1; i += 256) to[i] = reinterpret_cast<const uint4*>(sc)[i];
}

// Item: its request's first image (of chunk 0; those of the own pages' chunks
// follow the others), rows [r0, r0 + 128) and splits [sp0, sp1).
template <int HD>
__global__ void __launch_bounds__(Tc8Cfg<HD>::THREADS, 1) attn8_tc_kernel(Attn8Args a) {
  using C = Tc8Cfg<HD>;
  constexpr int KK = HD / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sq = smem;
  uint8_t* sk = sq + C::Q_BYTES;                   // unit u of K (KU per stage) at sk + (u % 2) * KU_BYTES; V of stage s at sv + (s % 2) * V_BYTES
  uint8_t* sv = sk + C::STAGES * C::KU_BYTES;
  uint8_t* so_out = sv + C::STAGES * C::V_BYTES;
  float* scales = reinterpret_cast<float*>(so_out + C::OUT_BYTES);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(scales) + C::SC_RING * C::SCALES);
  uint64_t* v_full = k_full + 2;     // [stage % 2] (and the two below)
  uint64_t* k_empty = v_full + 2;
  uint64_t* v_empty = k_empty + 2;
  uint64_t* s_full = v_empty + 2;    // [chunk % 2]: its 8-bit scores are there
  uint64_t* p_full = s_full + 2;     // its weights are, and O of the chunk before has been folded
  uint64_t* q_full = p_full + 2;
  uint64_t* s16_full = q_full + 1;   // scores of the own pages of a chunk that has some
  uint64_t* o_full = s16_full + 1;   // O of a chunk
  uint64_t* mma_done = o_full + 1;   // every MMA has completed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  __shared__ float2 ex[2][C::NT][128];  // [chunk % 2][half][row] Kv8Max of the chunk
  __shared__ float ex_l[2][C::NT][128];  // [chunk % 2] l of the halves at a split's end: the last two may be neighbours

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ int skip;
  const int half = blockIdx.x % C::HALVES, block_of = blockIdx.x / C::HALVES;
  const int kvh = block_of % a.Hkv;
  const int4 d0 = a.items[2 * (block_of / a.Hkv)], d1 = a.items[2 * (block_of / a.Hkv) + 1];
  const int image0 = d0.x, q0 = d0.y, qlen = d0.z, cached = d0.w, sp0 = d1.x, r0 = d1.y, sp1 = d1.z;
  const int G = a.Hq / a.Hkv, rows = qlen * G, kv_len = cached + qlen;
  const int r_end = min(rows, r0 + C::ROWS);
  const int p_min = cached + r0 / G, p_max = cached + (r_end - 1) / G;
  const int lo_min = a.window > 0 ? max(0, p_min - a.window + 1) : 0;
  const int own_lo = p_min >> 4, own_hi = p_max >> 4;
  const int ch0 = max(sp0 * (kSplit8 / kChunk8), lo_min / kChunk8);
  const int ch1 = min(sp1 * (kSplit8 / kChunk8) - 1, p_max / kChunk8);  // last chunk
  if (threadIdx.x == 0) {
    skip = a.status ? *reinterpret_cast<volatile int*>(a.status) : 0;
    for (int k = 0; k < 2; ++k) {
      mbar_init(&k_full[k], 1);
      mbar_init(&v_full[k], 1);
      mbar_init(&k_empty[k], 1);
      mbar_init(&v_empty[k], 1);
      mbar_init(&s_full[k], 1);
      mbar_init(&p_full[k], C::NS);
    }
    mbar_init(q_full, C::NS);
    mbar_init(s16_full, 1);
    mbar_init(o_full, 1);
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

  int issued_k = 0, issued_v = 0;  // units of K and stages of V whose copies have been issued (the copying thread's)
  if (warp < 4) {
    regs_dec<40>();
    if (warp == 0 && lane == 0) {
      const uint32_t id_s = idesc_f16(128, kChunk8), id_pv = idesc_f16(128, C::VD);
      const uint32_t q_lo = sw128_desc_lo(smem_u32(sq)), k_lo = sw128_desc_lo(smem_u32(sk)), v_lo = sw128_desc_lo(smem_u32(sv));
      auto wait = [&](uint64_t* f, int n) { return mbar_wait(f, n & 1, abort_flag, a.status); };
      // scores against the K of stage st into columns `col`, unit by unit
      auto scores = [&](int st, uint32_t col) -> bool {
#pragma unroll
        for (int part = 0; part < C::KU; ++part) {
          const int u = st * C::KU + part;
          if (!wait(&k_full[u & 1], u >> 1)) return false;
          tc_fence_after();
          const uint32_t k = k_lo + (u & 1) * (C::KU_BYTES >> 4);
          const uint32_t q = q_lo + part * (C::Q_BYTES / C::KU >> 4);
#pragma unroll
          for (int kk = 0; kk < KK / C::KU; ++kk)
            umma_bf16_lo(tmem + col, q + (kk >> 2) * (C::ROWS * 128 >> 4) + 2 * (kk & 3),
                         k + (kk >> 2) * (kChunk8 * 128 >> 4) + 2 * (kk & 3), id_s, part || kk ? 1u : 0u);
          umma_commit(&k_empty[u & 1]);
        }
        return true;
      };
      // O += weights of pages [x0, x1) in columns `p` times the V of stage st; first: from zero
      auto pv = [&](int st, uint32_t p, int x0, int x1, bool first) {
        const uint32_t v = v_lo + (st & 1) * (C::V_BYTES >> 4);
        auto one = [&](int x, uint32_t add) {
          umma_bf16_ta(tmem + 256, tmem + p + 8 * x, v + (x >> 2) * (C::VD * 128 >> 4) + 2 * (x & 3), id_pv, add);
        };
        if (first && x0 == 0 && x1 == kChunkPages) {
#pragma unroll
          for (int x = 0; x < kChunkPages; ++x) one(x, x ? 1u : 0u);
        } else {
#pragma unroll 1
          for (int x = x0; x < x1; ++x) one(x, first && x == x0 ? 0u : 1u);
        }
      };
      // Stages are numbered along the chunks: one for a chunk's 8-bit pages, one
      // more for its own pages.  Scores run up to two chunks ahead of P V; at
      // chunks with own pages, whose two stages fill both slots, they wait for
      // the P V of every chunk before.
      int ns = ch0, st_s = 0, st_v = 0;  // next chunk to score, its stage; the stage of the chunk whose P V is next
      bool ok = wait(q_full, 0);
#pragma unroll 1
      for (int ch = ch0 - 1; ok && ch <= ch1; ++ch) {  // (the first round only scores)
        if (ch >= ch0) {
          const int it = ch - ch0;
          const bool dg = diag(ch);
          ok = wait(&p_full[it & 1], it >> 1) && wait(&v_full[st_v & 1], st_v >> 1) &&
               (!dg || wait(&v_full[(st_v + 1) & 1], (st_v + 1) >> 1));
          if (!ok) break;
          tc_fence_after();
          const uint32_t p = 128 * (it & 1);
          pv(st_v, p, lo8(ch), hi8(ch), true);
          if (dg) pv(st_v + 1, p + 64, lo16(ch), hi16(ch), lo8(ch) >= hi8(ch));
          umma_commit(o_full);
          umma_commit(&v_empty[st_v & 1]);
          if (dg) umma_commit(&v_empty[(st_v + 1) & 1]);
          st_v += dg ? 2 : 1;
        }
#pragma unroll 1
        while (ns <= ch1 && ns <= ch + 2) {
          const bool dg = diag(ns);
          if (ns > ch + 1 && (dg || (ns > ch0 && diag(ns - 1)))) break;
          const int n = ns - ch0;
          ok = scores(st_s++, 128 * (n & 1));
          if (!ok) break;
          umma_commit(&s_full[n & 1]);
          if (dg) {  // own pages, into the other score buffer, which the next chunk takes later
            ok = scores(st_s++, 128 * (1 - (n & 1)));
            if (!ok) break;
            umma_commit(s16_full);
          }
          ++ns;
        }
      }
      umma_commit(mma_done);
    }
    if (warp == 1 && lane == 0) {  // ---- copies
      const int own_image = image0 + (kv_len + kChunk8 - 1) / kChunk8 - cached / kChunk8;  // + chunk: that of its own pages
      auto wait = [&](uint64_t* f, int n) { return mbar_wait(f, n & 1, abort_flag, a.status); };
      int st = 0;
      auto stage = [&](int image) -> bool {
        const uint8_t* src = a.images + (static_cast<size_t>(image) * a.Hkv + kvh) * C::IMAGE;
        const int s2 = st & 1;
#pragma unroll
        for (int part = 0; part < C::KU; ++part) {
          const int u = st * C::KU + part;
          if (u >= 2 && !wait(&k_empty[u & 1], (u >> 1) - 1)) return false;
          mbar_arrive_expect_tx(&k_full[u & 1], C::KU_BYTES + (part ? 0 : C::SCALES));
          bulk_load(sk + (u & 1) * C::KU_BYTES, src + part * C::KU_BYTES, C::KU_BYTES, &k_full[u & 1]);
          if (part == 0) bulk_load(scales + (st & 3) * (C::SCALES / 4), src + 2 * C::K_BYTES, C::SCALES, &k_full[u & 1]);
          issued_k = u + 1;
        }
        if (st >= 2 && !wait(&v_empty[s2], (st >> 1) - 1)) return false;
        mbar_arrive_expect_tx(&v_full[s2], C::V_BYTES);
        bulk_load(sv + s2 * C::V_BYTES, src + C::K_BYTES + half * C::V_BYTES, C::V_BYTES, &v_full[s2]);
        issued_v = ++st;
        return true;
      };
      bool ok = true;
#pragma unroll 1
      for (int ch = ch0; ok && ch <= ch1; ++ch) ok = stage(image0 + ch) && (!diag(ch) || stage(own_image + ch));
    }
  } else {
    // ---- softmax: two threads per row, of which thread h takes pages 4 h .. + 3 of a chunk and half of O's dims
    regs_inc<232>();
    constexpr int HP = kChunkPages / C::NT, OD = C::VD / C::NT;
    const int h = (warp - 4) >> 2, lr = (warp & 3) * 32 + lane, row = r0 + lr;
    const bool valid = row < r_end;
    const int tok = valid ? row / G : 0, hq = kvh * G + (valid ? row % G : 0);
    const int pos = valid ? cached + tok : -1, own = pos >> 4;
    const int lo = valid ? (a.window > 0 ? max(0, pos - a.window + 1) : 0) : 1;
    {  // the queries -> [hd block][row][64] fp16, 128-byte swizzle: 16 bytes per lane, whole rows per instruction
      constexpr int LPR = HD / 8, RPI = 32 / LPR;  // lanes of a row, rows of a warp's instruction
      const int w8 = warp - 4, c = lane % LPR;
      uint4 x[16 / RPI];
#pragma unroll
      for (int k = 0; k < 16 / RPI; ++k) {
        const int rr = r0 + w8 * 16 + k * RPI + lane / LPR;
        x[k] = rr < r_end ? reinterpret_cast<const uint4*>(a.q + (static_cast<size_t>(q0 + rr / G) * a.Hq + kvh * G + rr % G) * HD)[c]
                          : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int k = 0; k < 16 / RPI; ++k) {
        const int rl = w8 * 16 + k * RPI + lane / LPR;
        uint32_t mx = __vmaxu2(__vmaxu2(x[k].x & 0x7fff7fffu, x[k].y & 0x7fff7fffu), __vmaxu2(x[k].z & 0x7fff7fffu, x[k].w & 0x7fff7fffu));
#pragma unroll
        for (int d = 1; d < LPR; d *= 2) mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const int e = kv8_exp(kv8_max_halves(mx));
        const float up = kv8_up(e);
        if (c == 0) ex_l[0][0][rl] = e == 255 ? kv8_nan() : __fmul_rn(a.scale_log2, kv8_down(e));
        *reinterpret_cast<uint4*>(sq + (c >> 3) * (C::ROWS * 128) + rl * 128 + (((c & 7) ^ (rl & 7)) << 4)) =
            make_uint4(kv8_to_f16(x[k].x, up), kv8_to_f16(x[k].y, up), kv8_to_f16(x[k].z, up), kv8_to_f16(x[k].w, up));
      }
      fence_proxy_async_smem();
      mbar_arrive(q_full);
    }
    bool ok = softmax_sync<C::NS>(1, true);
    const float rowfac = ex_l[0][0][lr];
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    auto warp_wait = [&](uint64_t* f, int n) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(f, n & 1, abort_flag, a.status));
      return ok;
    };
    // The split in hand: this thread's l and O (pairs of dims); M, r: the running
    // maxima at the chunk whose weights were taken last, and O's exponent.  O of a chunk
    // is folded behind the next one's weights, with the factor for what is before it: 0
    // at a split's first chunk, as what O and L hold is then of another split, and
    // finite or NaN for good.
    Kv8Max M;
    float r = 0.f, L = 0.f;
    uint64_t O[OD / 2];
#pragma unroll
    for (int i = 0; i < OD / 2; ++i) O[i] = 0ull;
    const bool all = d1.w == kAttn8Folds;  // the run holds all of the block's splits: they are folded here
    float2 ml = make_float2(0.f, 0.f);  // maximum and l of those before, whose O is the totals
    bool have = false;
    int st = 0, n16 = 0;
    float al0 = 0.f, ao0 = 0.f, l0 = 0.f, S0 = 0.f, r0e = 0.f;  // of the chunk before: factors, l, largest score, exponent
#pragma unroll 1
    for (int ch = ch0; ch <= ch1 + 1; ++ch) {
      const int it = ch - ch0, pg0 = ch * kChunkPages + h * HP;  // this thread's first page
      const uint32_t s_at = lanes + 128 * (it & 1);
      float al = 0.f, ao = 0.f, l_ch = 0.f;
      if (ch <= ch1) {
        warp_wait(&s_full[it & 1], it >> 1);
        tc_fence_after();
        const float2* sc = reinterpret_cast<const float2*>(scales + (st & 3) * (C::SCALES / 4)) + h * HP;
        const float* so = scales + ((st + 1) & 3) * (C::SCALES / 4) + h * HP * 16;
        const bool dg = diag(ch);
        if (dg) {
          warp_wait(s16_full, n16++);
          tc_fence_after();
        }
        st += dg ? 2 : 1;
        // every row of the warp sees this half in 8 bits (rows that are none aside)
        const bool full = __all_sync(0xffffffffu, !valid || (lo <= pg0 * 16 && own >= pg0 + HP));
        float t[HP * 16], lv8[HP];
#pragma unroll
        for (int p0 = 0; p0 < HP; p0 += 2) {
          uint32_t x[32];
          ld32(s_at + 16 * (HP * h + p0), x);
          wait_ld32(x);
#pragma unroll
          for (int pg = p0; pg < p0 + 2; ++pg) {
            const float2 f = sc[pg];
            const float ks = __fmul_rn(f.x, rowfac);
            lv8[pg] = f.y;
            const uint64_t k2 = f2(ks, ks);
#pragma unroll
            for (int i = pg * 16; i < pg * 16 + 16; i += 2) {
              // (+ 0: a packed product and the difference below would come out as one fma)
              const uint64_t s2 = f2_fma(f2(x[i - 16 * p0], x[i - 16 * p0 + 1]), k2, 0ull);
              t[i] = f2_lo(s2);
              t[i + 1] = f2_hi(s2);
            }
          }
        }
        Kv8Max mc;  // of this half of the chunk
        if (!full) {
#pragma unroll
          for (int pg = 0; pg < HP; ++pg) {
            const int page = pg0 + pg;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (!(page < own && page * 16 + i >= lo)) t[pg * 16 + i] = -INFINITY;
            if (dg && page >= own_lo && page <= own_hi) {  // some rows' own page
              uint32_t y[16];
              ld16(lanes + 128 * (1 - (it & 1)) + 16 * (h * HP + pg), y);
              wait_ld16(y);
              if (page == own) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const int key = page * 16 + i;
                  const float v = __fmul_rn(__uint_as_float(y[i]), __fmul_rn(so[pg * 16 + i], rowfac));
                  if (key >= lo && key <= pos) t[pg * 16 + i] = v;
                  const float lv = so[kChunk8 + pg * 16 + i];
                  kv8_take(mc, t[pg * 16 + i], __fadd_rn(t[pg * 16 + i], lv));
                }
              }
            }
          }
        }
#pragma unroll
        for (int pg = 0; pg < HP; ++pg) {
          float m2[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 16; i += 2) m2[(i >> 1) & 1] = fmaxf(m2[(i >> 1) & 1], fmaxf(t[pg * 16 + i], t[pg * 16 + i + 1]));
          const float s1 = fmaxf(m2[0], m2[1]);
          if (full || pg0 + pg != own) kv8_take(mc, s1, __fadd_rn(s1, lv8[pg]));
        }
        ex[it & 1][h][lr] = make_float2(mc.s, mc.t);
        ok = softmax_sync<32 * C::NT>(2 + (warp & 3), ok);  // also: every score has been read
        if (!ok) break;
        const bool first = (ch & 3) == 0 || it == 0;
        if (first) {
          M = Kv8Max();
          r = 0.f;
        }
        const float s0 = M.s;
#pragma unroll
        for (int k = 0; k < C::NT; ++k) kv8_take(M, ex[it & 1][k][lr].x, ex[it & 1][k][lr].y);
        kv8_factors(M, s0, r, al, ao);
        if (first) al = ao = 0.f;
        const Kv8Base base(M, r);
        uint64_t l[4] = {0ull, 0ull, 0ull, 0ull};  // pair t: the partial sums (t, 0) and (t, 1)
        uint32_t pk[HP * 8];
        auto page_weights = [&](int pg, const Kv8Weight& w) {
          const uint64_t base2 = f2(w.base, w.base), back2 = f2(w.back, w.back);
#pragma unroll
          for (int i = pg * 8; i < pg * 8 + 8; ++i) {
            const uint64_t s2 = f2_sub(f2(t[2 * i], t[2 * i + 1]), base2);
            t[2 * i] = ex2(f2_lo(s2));
            t[2 * i + 1] = ex2(f2_hi(s2));
            pk[i] = pack_f16x2(t[2 * i], t[2 * i + 1]);
            l[i & 3] = f2_fma(f2(t[2 * i], t[2 * i + 1]), back2, l[i & 3]);
          }
        };
        if (full) {
#pragma unroll
          for (int pg = 0; pg < HP; ++pg) page_weights(pg, base(lv8[pg]));
        } else {
#pragma unroll
          for (int pg = 0; pg < HP; ++pg) {
            const int page = pg0 + pg;
            if (dg && page == own) {
#pragma unroll
              for (int i = pg * 8; i < pg * 8 + 8; ++i) {
                float back[2];
#pragma unroll
                for (int k = 2 * i; k < 2 * i + 2; ++k) {
                  // (a token that the row does not see stays out, whatever it holds)
                  const Kv8Weight w = t[k] != -INFINITY ? base(so[kChunk8 + k]) : kv8_no_weight();
                  t[k] = ex2(__fsub_rn(t[k], w.base));
                  back[k & 1] = w.back;
                }
                pk[i] = pack_f16x2(t[2 * i], t[2 * i + 1]);
                l[i & 3] = f2_fma(f2(t[2 * i], t[2 * i + 1]), f2(back[0], back[1]), l[i & 3]);
              }
            } else {  // (a page that the row does not see stays out, whatever its scale)
              const Kv8Weight w = page < own && page * 16 + 15 >= lo ? base(lv8[pg]) : kv8_no_weight();
              page_weights(pg, w);
            }
          }
        }
        if (dg) {  // the weights of own pages, 0 for the other rows, and 0 for them among the 8-bit pages
#pragma unroll
          for (int pg = 0; pg < HP; ++pg) {
            const int page = pg0 + pg;
            if (page < own_lo || page > own_hi) continue;
            uint32_t p16[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              p16[i] = page == own ? pk[pg * 8 + i] : 0u;
              pk[pg * 8 + i] = page == own ? 0u : pk[pg * 8 + i];
            }
            st8(s_at + 64 + 8 * (h * HP + pg), p16);
          }
        }
        st32(s_at + 8 * HP * h, pk);
        l_ch = __fadd_rn(__fadd_rn(__fadd_rn(f2_lo(l[0]), f2_hi(l[0])), __fadd_rn(f2_lo(l[1]), f2_hi(l[1]))),
                         __fadd_rn(__fadd_rn(f2_lo(l[2]), f2_hi(l[2])), __fadd_rn(f2_lo(l[3]), f2_hi(l[3]))));
      }
      if (it > 0) {  // O of the chunk before
        const int pc = ch - 1, sp = pc >> 2;
        warp_wait(o_full, it - 1);
        tc_fence_after();
        const uint64_t ao2 = f2(ao0, ao0);
#pragma unroll
        for (int c = 0; c < OD; c += 32) {
          uint32_t y[32];
          ld32(lanes + 256 + OD * h + c, y);
          wait_ld32(y);
#pragma unroll
          for (int i = 0; i < 16; ++i) O[c / 2 + i] = f2_fma(O[c / 2 + i], ao2, f2(y[2 * i], y[2 * i + 1]));
        }
        L = __fmaf_rn(L, al0, l0);
        if ((pc & 3) == 3 || pc == ch1) {  // the split's end
          ex_l[it & 1][h][lr] = L;
          ok = softmax_sync<32 * C::NT>(2 + (warp & 3), ok);
          if (!ok) break;
          float x[C::NT];
#pragma unroll
          for (int k = 0; k < C::NT; ++k) x[k] = ex_l[it & 1][k][lr];
          const float Ls = __fmul_rn(kv8_sum_parts(x), kPart), unit = ex2(__fadd_rn(r0e, kPartLog2));
          const uint64_t unit2 = f2(unit, unit);
          const bool sees = valid && max(lo, sp * kSplit8) <= min(pos, sp * kSplit8 + kSplit8 - 1);
          if (all) {
            // the totals with this split, in the merge kernel's arithmetic (what O holds is not needed after)
            const bool fold_in = sees && have;
            const float mn = fmaxf(ml.x, S0), ca = ex2(__fsub_rn(ml.x, mn)), cb = ex2(__fsub_rn(S0, mn));
            // (in scalars: the packed product and sum come out as one fma, which is not what the merge kernel computes)
            auto both = [&](uint32_t tot, float o) {
              const float t = __uint_as_float(tot);
              return fold_in ? __fadd_rn(__fmul_rn(t, ca), __fmul_rn(o, cb)) : have ? t : o;
            };
            const bool any = __any_sync(0xffffffffu, have), every = __all_sync(0xffffffffu, !valid || fold_in);
            if (sees) {
              ml = have ? make_float2(mn, __fadd_rn(__fmul_rn(ml.y, ca), __fmul_rn(Ls, cb))) : make_float2(S0, Ls);
            }
            uint4* to = reinterpret_cast<uint4*>(a.out + (static_cast<size_t>(q0 + tok) * a.Hq + hq) * HD + half * C::VD + OD * h);
#pragma unroll
            for (int c = 0; c < OD; c += 32) {
              uint32_t y[32];
              if (any) {
                ld32(lanes + 384 + OD * h + c, y);
                wait_ld32(y);
              }
              if (every) {
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  const uint64_t o = f2_fma(O[(c + i) / 2], unit2, 0ull);  // (kv8_part)
                  y[i] = __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(y[i]), ca), __fmul_rn(f2_lo(o), cb)));
                  y[i + 1] = __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(y[i + 1]), ca), __fmul_rn(f2_hi(o), cb)));
                }
              } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const uint64_t o = f2_fma(O[c / 2 + i], unit2, 0ull);
                  y[2 * i] = __float_as_uint(both(y[2 * i], f2_lo(o)));
                  y[2 * i + 1] = __float_as_uint(both(y[2 * i + 1], f2_hi(o)));
                }
              }
              if (pc < ch1) {
                st32(lanes + 384 + OD * h + c, y);
              } else if (valid) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  uint32_t w[4];
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    w[k] = pack_bf16x2(__fdiv_rn(__uint_as_float(y[8 * i + 2 * k]), ml.y), __fdiv_rn(__uint_as_float(y[8 * i + 2 * k + 1]), ml.y));
                  to[c / 8 + i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
              }
            }
            have = have || sees;
            tmem_wait_st();
          } else {
            // The split's partial.  OUT_DIMS at a time go through shared memory, so
            // that a store of the warp writes as many of a few rows each.
            if (sees && h == 0 && half == 0) {
              const size_t base = (static_cast<size_t>(d1.w + tok) * a.Hq + hq) * a.max_splits + sp;
              a.part_ml[base * 2] = S0;
              a.part_ml[base * 2 + 1] = Ls;
            }
            float4* buf = reinterpret_cast<float4*>(so_out) + (warp - 4) * (8 * C::OUT_DIMS);  // [row][W], the 16-byte words XORed with the row
            const unsigned rows_seen = __ballot_sync(0xffffffffu, sees);
#pragma unroll
            for (int c = 0; c < OD; c += C::OUT_DIMS) {
              constexpr int W = C::OUT_DIMS / 4;  // words of a row
#pragma unroll
              for (int i = 0; i < W; ++i) {
                const uint64_t v0 = f2_fma(O[c / 2 + 2 * i], unit2, 0ull), v1 = f2_fma(O[c / 2 + 2 * i + 1], unit2, 0ull);
                buf[lane * W + (i ^ (lane & (W - 1)))] = make_float4(f2_lo(v0), f2_hi(v0), f2_lo(v1), f2_hi(v1));
              }
              __syncwarp();
#pragma unroll
              for (int k = 0; k < W; ++k) {
                const int rl = k * (32 / W) + lane / W, i = lane % W;
                if ((rows_seen >> rl) & 1u) {
                  const int rr = r0 + (warp & 3) * 32 + rl;
                  const size_t base = (static_cast<size_t>(d1.w + rr / G) * a.Hq + kvh * G + rr % G) * a.max_splits + sp;
                  *reinterpret_cast<float4*>(a.part_o + base * HD + half * C::VD + OD * h + c + i * 4) = buf[rl * W + (i ^ (rl & (W - 1)))];
                }
              }
              __syncwarp();
            }
          }
        }
      }
      if (ch <= ch1) {
        al0 = al;
        ao0 = ao;
        l0 = l_ch;
        S0 = M.s;
        r0e = r;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[it & 1]);
      }
    }
  }
  // Teardown: copies land and issued MMAs finish, then tensor memory is freed.
  if (warp == 1 && lane == 0) {
    for (int u = max(0, issued_k - 2); u < issued_k; ++u) drain_wait(&k_full[u & 1], (u >> 1) & 1);
    for (int st = max(0, issued_v - 2); st < issued_v; ++st) drain_wait(&v_full[st & 1], (st >> 1) & 1);
  }
  if (warp == 0 && lane == 0) drain_wait(mma_done, 0);
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int HD, int FMT>
int launch_attn8_tc_t(const Attn8Args& a, int n_chunks, int n_blocks, cudaStream_t s) {
  using C = Tc8Cfg<HD>;
  constexpr int kExpandSmem = 1024 + C::K_BYTES + C::SCALES;
  VD_CUDA_TRY(cudaFuncSetAttribute(attn8_expand_kernel<HD, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kExpandSmem));
  VD_CUDA_TRY(launch_k(attn8_expand_kernel<HD, FMT>, dim3(static_cast<unsigned>(n_chunks) * a.Hkv * 2), dim3(256), kExpandSmem, s, a));
  VD_CUDA_TRY(cudaFuncSetAttribute(attn8_tc_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM));
  VD_CUDA_TRY(launch_k(attn8_tc_kernel<HD>, dim3(static_cast<unsigned>(n_blocks) * a.Hkv * C::HALVES), dim3(C::THREADS), C::SMEM, s, a));
  return VD_OK;
}

}  // namespace

size_t attn8_image_bytes(int hd) { return hd == 64 ? Tc8Cfg<64>::IMAGE : hd == 128 ? Tc8Cfg<128>::IMAGE : Tc8Cfg<256>::IMAGE; }

int launch_attention8_tc(const Attn8Args& a, int hd, int format, int n_chunks, int n_blocks, cudaStream_t s) {
  if (n_blocks <= 0) return VD_OK;
  const bool i8 = format == VD_KV8_INT8;
  if (hd == 64)
    return i8 ? launch_attn8_tc_t<64, kKv8Int8>(a, n_chunks, n_blocks, s) : launch_attn8_tc_t<64, kKv8E4m3>(a, n_chunks, n_blocks, s);
  if (hd == 128)
    return i8 ? launch_attn8_tc_t<128, kKv8Int8>(a, n_chunks, n_blocks, s) : launch_attn8_tc_t<128, kKv8E4m3>(a, n_chunks, n_blocks, s);
  if (hd == 256)
    return i8 ? launch_attn8_tc_t<256, kKv8Int8>(a, n_chunks, n_blocks, s) : launch_attn8_tc_t<256, kKv8E4m3>(a, n_chunks, n_blocks, s);
  return fail(VD_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
}

}  // namespace vd
