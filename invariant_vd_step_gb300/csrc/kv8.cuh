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
// 8-bit ones, which carry the V scales in the product, have like sizes in fp16.  (Rows whose
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

// What a row's weights are taken relative to, over the keys seen so far: its largest
// score s, and the largest t of t_j = s_j + log2 of j's V scale.  Maxima, so that they
// do not depend on the order of the keys; they ignore NaN (whose weights are NaN).
struct Kv8Max {
  float s = -INFINITY, t = -INFINITY;
};
__device__ __forceinline__ void kv8_take(Kv8Max& m, float s, float t) {
  m.s = fmaxf(m.s, s);
  m.t = fmaxf(m.t, t);
}
// r, the exponent of O: O holds 2^-r of the values' sum, so that the largest of the
// weights times V scales that enter the product in fp16 is about 1.  Where scores are so
// large that t has lost the V scale, r is still within the scales' range.
__device__ __forceinline__ float kv8_exponent(const Kv8Max& m) {
  return m.s == -INFINITY ? 0.f : fminf(fmaxf(__fsub_rn(m.t, m.s), -94.f), 122.f);
}
// m has taken up a chunk: the factors for the l and the O before it, of base s0 and
// exponent r, which becomes m's.
__device__ __forceinline__ void kv8_factors(const Kv8Max& m, float s0, float& r, float& al, float& ao) {
  const float d = m.s == s0 ? 0.f : __fsub_rn(s0, m.s), r0 = r;
  r = kv8_exponent(m);
  al = ex2(d);
  ao = ex2(__fadd_rn(d, __fsub_rn(r0, r)));
}
// A key whose V scale has the log2 lv enters the product with 2^(s_j - base), base = s -
// (lv - r): its weight times 2^(lv - r), in one exponential; l takes that times back,
// 2^(r - lv).  lv - r counts as -90 below, where nothing is left in fp16 either way and
// weights above 2^-36 still are normal numbers.  (NaN stays.)
struct Kv8Weight {
  float base, back;
};
struct Kv8Base {  // of a row at a chunk; s: any value where no key has been seen (every score is -inf then)
  float s, r, k;
  // k: 0 where float32 scores are 16 or more apart (2^27): there the base is s, as its
  // rounding would move what should be about 1 out of fp16's range
  __device__ __forceinline__ Kv8Base(const Kv8Max& m, float r_)
      : s(m.s == -INFINITY ? 0.f : m.s), r(r_), k(fabsf(m.s) < 0x1p27f ? -1.f : 0.f) {}
  __device__ __forceinline__ Kv8Base() : s(0.f), r(0.f), k(0.f) {}
  __device__ __forceinline__ Kv8Weight operator()(float lv) const {
    float up = __fsub_rn(lv, r);
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(up) : "f"(up), "f"(-90.f));
    return {__fmaf_rn(up, k, s), ex2(-up)};
  }
};
__device__ __forceinline__ Kv8Weight kv8_no_weight() { return {0.f, 0.f}; }  // of keys whose scores are -inf

// A split's partial: base s, l 2^-24 and the sum of the values 2^-24, which float32 holds
// for any bf16 values (2^24 of them at 2^128) and at any scale above 2^-94.
constexpr float kPartLog2 = -24.f, kPart = 0x1p-24f;
__device__ __forceinline__ float kv8_part(float o, float unit) {
  return __fmaf_rn(o, unit, 0.f);  // (+ 0: a zero of O may have either sign, by the kernel that ran)
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
