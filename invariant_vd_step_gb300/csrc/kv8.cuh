// The 8-bit KV cache on the device: page layout, codes and the exponents that
// bring bf16 rows into fp16 without rounding.
#pragma once

#include "vd_device.cuh"

namespace vd {

constexpr int kKv8Int8 = 0, kKv8E4m3 = 1;
constexpr int kChunkParts = 2;  // parts of a chunk's pages whose l are summed apart (threads per row of the tcgen05 kernel)

// Codes of one (page, head): K part, then V part, each HD / 32 units of 512
// bytes: 16 bytes for each lane of a warp, the operand words of mma.sync
// m16n8k16 (vd_kv8.h has the formula).  Word w of a lane (g = lane / 4, t = lane
// % 4): in K, k-step w / 2 of 16 dims and key block w % 2 of 8 keys, the codes of
// key g at dims 2t, 2t + 1, 2t + 8, 2t + 9; in V, dim 8 w + g of keys 2t, 2t + 1,
// 2t + 8, 2t + 9.  A warp then reads a page in whole 16-byte words and turns it
// into operands without shared memory traffic beyond that, without bank
// conflicts and without a shuffle.
template <int HD>
struct Kv8Cfg {
  static constexpr int PART = 16 * HD;
  static constexpr int UNITS = HD / 32;
};

// Four codes -> two fp16 pairs, exactly.  int8 (stored plus 128): the bytes
// become the low bits of 1024 + u, from which 1152 is subtracted.
template <int FMT>
__device__ __forceinline__ void kv8_expand(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == kKv8Int8) {
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
  } else {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

// A bf16 row (a query, or a token of the page being filled) enters the fp16
// products times 2^n, with n such that its largest magnitude, whose bits without
// the sign are `amax`, lands in [2^7, 2^8): exact for every element above 2^-24
// of it (fp16 has 11 bits, bf16 8), off by 2^-32 of the largest below.  The range
// is that of the codes, so that the weights of the own page's tokens and of the
// 8-bit ones, which carry the V scales, have like sizes in fp16.  (Rows whose
// largest is below 2^-87 count from there.)
__device__ __forceinline__ int kv8_exp(uint32_t amax) { return max(static_cast<int>(amax >> 7), 40); }  // 255: inf or NaN
__device__ __forceinline__ float kv8_up(int e) { return __uint_as_float(static_cast<uint32_t>(261 - e) << 23); }  // 2^n
__device__ __forceinline__ float kv8_down(int e) { return __uint_as_float(static_cast<uint32_t>(e - 7) << 23); }  // 2^-n
__device__ __forceinline__ float kv8_log2_down(int e) { return static_cast<float>(e - 134); }                     // -n
__device__ __forceinline__ float kv8_nan() { return __uint_as_float(0x7fc00000u); }
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two bf16 values of one row times f, as fp16.
__device__ __forceinline__ uint32_t kv8_to_f16(uint32_t v, float f) {
  return pack_f16x2(__fmul_rn(bf16_lo(v), f), __fmul_rn(bf16_hi(v), f));
}
__device__ __forceinline__ uint32_t kv8_max_halves(uint32_t v) { return max(v & 0xffffu, v >> 16); }

// The running maximum m of a row after a chunk whose largest score is mx, and the
// factor for the sums before it (1 where it stays, -inf included).
__device__ __forceinline__ void kv8_running_max(float& m, float mx, float& alpha) {
  const float mn = fmaxf(m, mx);
  alpha = mn == m ? 1.0f : ex2(__fsub_rn(m, mn));
  m = mn;
}

__device__ __forceinline__ float kv8_sum_parts(const float (&x)[kChunkParts]) {
  float s = 0.f;
  if constexpr (kChunkParts == 2) s = __fadd_rn(x[0], x[1]);
  if constexpr (kChunkParts == 4) s = __fadd_rn(__fadd_rn(x[0], x[1]), __fadd_rn(x[2], x[3]));
  return s;
}

__device__ __forceinline__ void mma_f16_16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Untiled bulk copy, global to shared (both 16-byte aligned, bytes a multiple of 16).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
}  // namespace vd
