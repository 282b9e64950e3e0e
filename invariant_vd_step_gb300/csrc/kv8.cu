// Pages of the 8-bit KV cache: sealing bf16 pages into it, opening them again,
// and copies of pages within a pool or cache.  All three move bytes and are bound
// by memory once a call holds a few thousand (page, layer, head) blocks; below
// that by the launch.
#include <cuda_fp16.h>

#include "kv8.cuh"
#include "vd_internal.h"

namespace vd {
namespace {

template <typename P>
__device__ __forceinline__ int2 pair_of(const P& p, int i) {
  return p.dev ? p.dev[i] : p.at[i];
}

constexpr float kKv8Least = 8.271806125530277e-25f;  // 2^-80: blocks below it count from there

// Codes of values x of a block with largest magnitude a: the exact quotient top x /
// a, rounded once.
//
// e4m3: with s the power of two that brings a into [1, 2), x s top is exact (bf16 has
// 8 bits, 448 has 3).  y0 = x s top r with r = 1 / (a s) rounded is off by at most
// 2^-23 of itself; y = y0 + (x s top - y0 a s) r, the residual exact in an fma
// (Markstein's correction of a quotient), is the quotient itself wherever float32
// holds it, as it does at every tie of the codes' rounding, and else off by far less
// than the 2^-16 of itself that separates a quotient that is no tie from the next one.
//
// int8: one fma per value, x c + 1.5 * 2^23 + 128 with c = 127 / a rounded up, whose
// low byte is the code.  A quotient that is no tie is 2^-9 or more from one, c's error
// moves it by less than 2^-16.  127 x / a = n + 1/2 with 8-bit significands means that
// |x| = a / 2 (127 is prime), where 63.5 and a little more both round to 64, as the
// tie does; or that a's significand is 127, where c is a power of two and exact.
//
// Sealing and opening 512 pages of 32 layers, 8 heads of 128, e4m3: 520 us, 6.2 TB/s;
// with a division per value, and stores that met a bank up to eight times, 647.
struct Kv8Quotient {
  float m, a, r;  // e4m3: s top, a s, r; int8: r is c
};
template <int FMT>
__device__ __forceinline__ Kv8Quotient kv8_quotient(float amax) {
  if constexpr (FMT == kKv8Int8) return {0.f, 0.f, __fdiv_ru(127.0f, amax)};
  const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;  // [-80, 127]
  // 2^-e in two factors, as 2^-127 is below the normal numbers
  const float s0 = __uint_as_float(static_cast<uint32_t>(127 - e / 2) << 23);
  const float s1 = __uint_as_float(static_cast<uint32_t>(127 - (e - e / 2)) << 23);
  Kv8Quotient q;
  q.a = __fmul_rn(__fmul_rn(amax, s0), s1);
  q.m = __fmul_rn(__fmul_rn(448.0f, s0), s1);
  q.r = __frcp_rn(q.a);
  return q;
}
__device__ __forceinline__ float kv8_divide(const Kv8Quotient& q, float x) {
  const float xs = __fmul_rn(x, q.m), y0 = __fmul_rn(xs, q.r);
  return __fmaf_rn(__fmaf_rn(-y0, q.a, xs), q.r, y0);
}
template <int FMT>
__device__ __forceinline__ uint32_t kv8_code4(const Kv8Quotient& q, float x0, float x1, float x2, float x3) {
  if constexpr (FMT == kKv8Int8) {
    const float x[4] = {x0, x1, x2, x3};
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(__fmaf_rn(x[i], q.r, 12582912.0f + 128.0f));
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  } else {
    const float y[4] = {kv8_divide(q, x0), kv8_divide(q, x1), kv8_divide(q, x2), kv8_divide(q, x3)};
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y[1]), "f"(y[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y[3]), "f"(y[2]));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  }
}

// One warp per (pair, layer, head, K or V).  An item of a lane is 64 bytes of the
// page and 32 of the codes: of K, a k-step of the tokens r and r + 8; of V, 8 dims of
// the tokens 2t, 2t + 1, 2t + 8, 2t + 9.  Either way its codes are whole operand
// words, which go through shared memory so that both sides move in order.  There 16
// bytes of a KB trade places so that a warp's stores meet no bank twice.
template <int HD>
struct SealItem {
  int token, chunk;  // of 16 bytes v of the item
  static __device__ __forceinline__ SealItem at(int kv, int idx, int v) {
    if (kv) return {2 * (idx / (HD / 8)) + (v & 1) + 8 * (v >> 1), idx % (HD / 8)};
    return {(idx & 7) + 8 * (v >> 1), 2 * (idx >> 3) + (v & 1)};
  }
};
// places of 16 bytes i of KB j
template <int HD>
__device__ __forceinline__ int seal_place(int kv, int j, int i) {
  return j * 32 + (kv ? i ^ ((j * (256 / HD)) & 7) : i ^ ((i >> 3) & 3));
}
template <int HD>
__device__ __forceinline__ int seal_word_v(int c, int g, int t) {  // dim 8 c + g, tokens 2t ..
  return seal_place<HD>(1, c >> 2, g * 4 + t) * 4 + (c & 3);
}
template <int HD>
__device__ __forceinline__ int seal_pair_k(int kk, int r, int t) {  // dims 16 kk + 2t .., tokens r, r + 8
  return seal_place<HD>(0, kk >> 1, r * 4 + t) * 2 + (kk & 1);
}

template <int HD, int FMT, typename P>
__global__ void __launch_bounds__(128) kv8_seal_kernel(SealArgs a, const __grid_constant__ P pairs) {
  constexpr int PART = Kv8Cfg<HD>::PART, IT = HD / 64;
  __shared__ uint4 stage[4][PART / 16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const long long unit = static_cast<long long>(blockIdx.x) * 4 + warp;
  const int kv = static_cast<int>(unit & 1), per = 2 * a.Hkv * a.layers;
  if (unit >= static_cast<long long>(pairs.n) * per) return;
  const int i = static_cast<int>(unit / per), rest = static_cast<int>(unit % per) >> 1;
  const int head = rest % a.Hkv, layer = rest / a.Hkv;
  const int2 pp = pair_of(pairs, i);
  const __nv_bfloat16* src = a.pool + layer * a.pool_layer + ((static_cast<long long>(pp.x) * 2 + kv) * a.Hkv + head) * PART;
  const long long block = static_cast<long long>(pp.y) * a.Hkv + head;
  uint8_t* dst = a.codes + layer * a.codes_layer + block * (2 * PART) + kv * PART;
  uint4 x[IT][4];
#pragma unroll
  for (int it = 0; it < IT; ++it)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const auto at = SealItem<HD>::at(kv, it * 32 + lane, v);
      x[it][v] = *reinterpret_cast<const uint4*>(src + at.token * HD + at.chunk * 8);
    }
  uint32_t mx = 0u;
#pragma unroll
  for (int it = 0; it < IT; ++it)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const uint4 y = x[it][v];
      mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(y.x & 0x7fff7fffu, y.y & 0x7fff7fffu), __vmaxu2(y.z & 0x7fff7fffu, y.w & 0x7fff7fffu)));
    }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, d));
  const uint32_t mb = kv8_max_halves(mx);
  const bool finite = mb < 0x7f80u;
  const float amax = finite ? fmaxf(__uint_as_float(mb << 16), kKv8Least) : 1.0f;
  const Kv8Quotient q = kv8_quotient<FMT>(amax);
  if (!finite) {  // its codes are those of zeros
#pragma unroll
    for (int it = 0; it < IT; ++it)
#pragma unroll
      for (int v = 0; v < 4; ++v) x[it][v] = make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int idx = it * 32 + lane;
    const uint32_t* w[4] = {&x[it][0].x, &x[it][1].x, &x[it][2].x, &x[it][3].x};
    if (kv) {
      uint32_t* words = reinterpret_cast<uint32_t*>(stage[warp]);
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        float f[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) f[v] = (g & 1) ? bf16_hi(w[v][g >> 1]) : bf16_lo(w[v][g >> 1]);
        words[seal_word_v<HD>(idx % (HD / 8), g, idx / (HD / 8))] = kv8_code4<FMT>(q, f[0], f[1], f[2], f[3]);
      }
    } else {
      uint2* words = reinterpret_cast<uint2*>(stage[warp]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {  // dims 2 t, + 1, + 8, + 9 of both tokens
        uint32_t c[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t y0 = w[2 * h][t], y1 = w[2 * h + 1][t];
          c[h] = kv8_code4<FMT>(q, bf16_lo(y0), bf16_hi(y0), bf16_lo(y1), bf16_hi(y1));
        }
        words[seal_pair_k<HD>(idx >> 3, idx & 7, t)] = make_uint2(c[0], c[1]);
      }
    }
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < PART / 512; ++j) reinterpret_cast<uint4*>(dst)[j * 32 + lane] = stage[warp][seal_place<HD>(kv, j, lane)];
  if (lane == 0) {
    float* sc = reinterpret_cast<float*>(a.scales + layer * a.scales_layer + block);
    const float scale = finite ? __fdiv_rn(amax, FMT == kKv8Int8 ? 127.0f : 448.0f) : kv8_nan();
    if (!kv) {
      sc[0] = scale;
    } else {
      sc[1] = __frcp_rn(scale);
      sc[2] = log2f(scale);
      sc[3] = scale;
    }
  }
}

template <int HD, int FMT, typename P>
__global__ void __launch_bounds__(128) kv8_unseal_kernel(SealArgs a, const __grid_constant__ P pairs) {
  constexpr int PART = Kv8Cfg<HD>::PART, IT = HD / 64;
  __shared__ uint4 stage[4][PART / 16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const long long unit = static_cast<long long>(blockIdx.x) * 4 + warp;
  const int kv = static_cast<int>(unit & 1), per = 2 * a.Hkv * a.layers;
  if (unit >= static_cast<long long>(pairs.n) * per) return;
  const int i = static_cast<int>(unit / per), rest = static_cast<int>(unit % per) >> 1;
  const int head = rest % a.Hkv, layer = rest / a.Hkv;
  const int2 pp = pair_of(pairs, i);
  const long long block = static_cast<long long>(pp.x) * a.Hkv + head;
  const uint8_t* src = a.codes + layer * a.codes_layer + block * (2 * PART) + kv * PART;
  __nv_bfloat16* dst = a.pool + layer * a.pool_layer + ((static_cast<long long>(pp.y) * 2 + kv) * a.Hkv + head) * PART;
  const float4 sc = a.scales[layer * a.scales_layer + block];
  const float scale = kv ? sc.w : sc.x;
#pragma unroll
  for (int j = 0; j < PART / 512; ++j) stage[warp][seal_place<HD>(kv, j, lane)] = reinterpret_cast<const uint4*>(src)[j * 32 + lane];
  __syncwarp();
  auto value2 = [&](uint32_t h) {  // fp16 pair of codes -> bf16 pair of values
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_bf16x2(__fmul_rn(f.x, scale), __fmul_rn(f.y, scale));
  };
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int idx = it * 32 + lane;
    uint32_t y[4][4];
    if (kv) {
      const uint32_t* words = reinterpret_cast<const uint32_t*>(stage[warp]);
      const int t = idx / (HD / 8), c = idx % (HD / 8);
#pragma unroll
      for (int g = 0; g < 8; g += 2) {  // dims 8 c + g, + 1 of tokens 2t, 2t + 1, 2t + 8, 2t + 9
        uint32_t lo0, hi0, lo1, hi1;
        kv8_expand<FMT>(words[seal_word_v<HD>(c, g, t)], lo0, hi0);
        kv8_expand<FMT>(words[seal_word_v<HD>(c, g + 1, t)], lo1, hi1);
        y[0][g >> 1] = value2(__byte_perm(lo0, lo1, 0x5410));
        y[1][g >> 1] = value2(__byte_perm(lo0, lo1, 0x7632));
        y[2][g >> 1] = value2(__byte_perm(hi0, hi1, 0x5410));
        y[3][g >> 1] = value2(__byte_perm(hi0, hi1, 0x7632));
      }
    } else {
      const uint2* words = reinterpret_cast<const uint2*>(stage[warp]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint2 w = words[seal_pair_k<HD>(idx >> 3, idx & 7, t)];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t lo, hi;
          kv8_expand<FMT>(h ? w.y : w.x, lo, hi);
          y[2 * h][t] = value2(lo);
          y[2 * h + 1][t] = value2(hi);
        }
      }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const auto at = SealItem<HD>::at(kv, idx, v);
      *reinterpret_cast<uint4*>(dst + at.token * HD + at.chunk * 8) = make_uint4(y[v][0], y[v][1], y[v][2], y[v][3]);
    }
  }
}

// One block of 256 threads moves 16 KB of a page: four 16-byte words per thread,
// all loaded before the first is stored.  700 pages of the 8-bit cache, 32 layers of
// 8 heads of 128: 218 us, 6.7 TB/s, what a copy reaches.
constexpr int kCopyBlock = 16384;
template <typename P>
__global__ void __launch_bounds__(256) copy_pages_kernel(CopyArgs a, const __grid_constant__ P pairs, int parts) {
  pdl_wait();
  pdl_trigger();
  const int part = blockIdx.x % parts, rest = blockIdx.x / parts;
  const int layer = rest % a.layers;
  const int2 pp = pair_of(pairs, rest / a.layers);
  const uint8_t* src = a.data + layer * a.layer + pp.x * a.bytes;
  uint8_t* dst = a.data + layer * a.layer + pp.y * a.bytes;
  uint4 v[4];
  const long long at = static_cast<long long>(part) * kCopyBlock + threadIdx.x * 16;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (at + k * 4096 < a.bytes) v[k] = *reinterpret_cast<const uint4*>(src + at + k * 4096);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (at + k * 4096 < a.bytes) *reinterpret_cast<uint4*>(dst + at + k * 4096) = v[k];
  if (part == 0)
    for (int k = threadIdx.x; k < a.n_extra; k += 256) {
      float4* e = a.extra + layer * a.extra_layer;
      e[static_cast<long long>(pp.y) * a.n_extra + k] = e[static_cast<long long>(pp.x) * a.n_extra + k];
    }
}

template <int HD, typename P>
int launch_seal_t(const SealArgs& a, const P& p, bool unseal, cudaStream_t s) {
  const long long units = static_cast<long long>(p.n) * a.layers * a.Hkv * 2;
  const dim3 grid(static_cast<unsigned>((units + 3) / 4));
  const bool i8 = a.format == VD_KV8_INT8;
  auto k = unseal ? (i8 ? kv8_unseal_kernel<HD, kKv8Int8, P> : kv8_unseal_kernel<HD, kKv8E4m3, P>)
                  : (i8 ? kv8_seal_kernel<HD, kKv8Int8, P> : kv8_seal_kernel<HD, kKv8E4m3, P>);
  VD_CUDA_TRY(launch_k(k, grid, dim3(128), 0, s, a, p));
  return VD_OK;
}

template <typename P>
int launch_seal_p(const SealArgs& a, const P& p, bool unseal, cudaStream_t s) {
  if (p.n <= 0) return VD_OK;
  if (a.hd == 64) return launch_seal_t<64>(a, p, unseal, s);
  if (a.hd == 128) return launch_seal_t<128>(a, p, unseal, s);
  if (a.hd == 256) return launch_seal_t<256>(a, p, unseal, s);
  return fail(VD_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
}
template <typename P>
int launch_copy_p(const CopyArgs& a, const P& p, cudaStream_t s) {
  if (p.n <= 0) return VD_OK;
  const int parts = static_cast<int>((a.bytes + kCopyBlock - 1) / kCopyBlock);
  VD_CUDA_TRY(launch_k(copy_pages_kernel<P>, dim3(static_cast<unsigned>(p.n * a.layers * parts)), dim3(256), 0, s, a, p, parts));
  return VD_OK;
}

}  // namespace

int launch_kv8_seal(const SealArgs& a, const PagePairs& p, bool unseal, cudaStream_t s) { return launch_seal_p(a, p, unseal, s); }
int launch_kv8_seal(const SealArgs& a, const ManyPagePairs& p, bool unseal, cudaStream_t s) { return launch_seal_p(a, p, unseal, s); }
int launch_copy_pages(const CopyArgs& a, const PagePairs& p, cudaStream_t s) { return launch_copy_p(a, p, s); }
int launch_copy_pages(const CopyArgs& a, const ManyPagePairs& p, cudaStream_t s) { return launch_copy_p(a, p, s); }

}  // namespace vd
