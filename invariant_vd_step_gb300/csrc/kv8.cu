// Pages of the 8-bit KV cache: sealing bf16 pages into it, opening them again,
// and copies of pages within a pool or cache.  All three move bytes and are bound
// by memory once a call holds a few thousand (page, layer, head) blocks; below
// that by the launch.
#include <cuda_fp16.h>

#include "kv8.cuh"
#include "vd_internal.h"

namespace vd {
namespace {

__device__ __forceinline__ int2 pair_of(const PagePairs& p, int i) { return p.dev ? p.dev[i] : p.at[i]; }

constexpr float kKv8Least = 8.271806125530277e-25f;  // 2^-80: blocks below it count from there

// The codes of two values, in the low 16 bits.  127 x and 7 x are exact (bf16 has
// 8 bits) and the division is rounded once, and a quotient that is no tie is at
// least 2^-13 of it away from one, so the code is the rounding of the exact
// quotient; the factor 64 of e4m3's 448 = 7 * 64 is exact.
template <int FMT>
__device__ __forceinline__ uint32_t kv8_code2(float x0, float x1, float a) {
  if constexpr (FMT == kKv8Int8) {
    const int q0 = __float2int_rn(__fdiv_rn(__fmul_rn(x0, 127.0f), a));
    const int q1 = __float2int_rn(__fdiv_rn(__fmul_rn(x1, 127.0f), a));
    return static_cast<uint32_t>(q0 + 128) | (static_cast<uint32_t>(q1 + 128) << 8);
  } else {
    const float y0 = __fmul_rn(__fdiv_rn(__fmul_rn(x0, 7.0f), a), 64.0f);
    const float y1 = __fmul_rn(__fdiv_rn(__fmul_rn(x1, 7.0f), a), 64.0f);
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y1), "f"(y0));
    return r;
  }
}
template <int FMT>
__device__ __forceinline__ uint32_t kv8_code_zero() {
  return FMT == kKv8Int8 ? 0x80808080u : 0u;
}

// One warp per (pair, layer, head, K or V).  Its lanes' items: of K, a token's 32
// bytes of one k-step; of V, 16 bytes of the four tokens 2t, 2t + 1, 2t + 8, 2t + 9.
// Either way an item's codes are whole operand words, which go to their place in
// shared memory and leave it in order.
template <int HD, int FMT>
__global__ void __launch_bounds__(128) kv8_seal_kernel(SealArgs a, const __grid_constant__ PagePairs pairs) {
  constexpr int PART = Kv8Cfg<HD>::PART, IT = HD / 64;  // V items (of 64 bytes) per lane; K has twice as many, of 32
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
      int token, chunk;
      if (kv) {
        const int idx = it * 32 + lane, t = idx / (HD / 8);
        token = 2 * t + (v & 1) + 8 * (v >> 1);
        chunk = idx % (HD / 8);
      } else {
        const int idx = (2 * it + (v >> 1)) * 32 + lane;
        token = idx / (HD / 16);
        chunk = 2 * (idx % (HD / 16)) + (v & 1);
      }
      x[it][v] = *reinterpret_cast<const uint4*>(src + token * HD + chunk * 8);
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
  const float amax = fmaxf(__uint_as_float(mb << 16), kKv8Least);
  uint32_t* words = reinterpret_cast<uint32_t*>(stage[warp]);
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const uint32_t* w[4] = {&x[it][0].x, &x[it][1].x, &x[it][2].x, &x[it][3].x};
    if (kv) {
      const int idx = it * 32 + lane, t = idx / (HD / 8), c = idx % (HD / 8);
#pragma unroll
      for (int g = 0; g < 8; ++g) {  // dim 8 c + g of the four tokens
        float f[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) f[v] = (g & 1) ? bf16_hi(w[v][g >> 1]) : bf16_lo(w[v][g >> 1]);
        words[(c >> 2) * 128 + (g * 4 + t) * 4 + (c & 3)] =
            finite ? kv8_code2<FMT>(f[0], f[1], amax) | (kv8_code2<FMT>(f[2], f[3], amax) << 16) : kv8_code_zero<FMT>();
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int idx = (2 * it + h) * 32 + lane, token = idx / (HD / 16), kk = idx % (HD / 16);
#pragma unroll
        for (int t = 0; t < 4; ++t) {  // dims 16 kk + 2 t, + 1, + 8, + 9
          const uint32_t y0 = w[2 * h][t], y1 = w[2 * h + 1][t];
          words[(kk >> 1) * 128 + ((token & 7) * 4 + t) * 4 + (kk & 1) * 2 + (token >> 3)] =
              finite ? kv8_code2<FMT>(bf16_lo(y0), bf16_hi(y0), amax) | (kv8_code2<FMT>(bf16_lo(y1), bf16_hi(y1), amax) << 16)
                     : kv8_code_zero<FMT>();
        }
      }
    }
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < PART / 512; ++j) reinterpret_cast<uint4*>(dst)[j * 32 + lane] = stage[warp][j * 32 + lane];
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

template <int HD, int FMT>
__global__ void __launch_bounds__(128) kv8_unseal_kernel(SealArgs a, const __grid_constant__ PagePairs pairs) {
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
  for (int j = 0; j < PART / 512; ++j) stage[warp][j * 32 + lane] = reinterpret_cast<const uint4*>(src)[j * 32 + lane];
  __syncwarp();
  const uint32_t* words = reinterpret_cast<const uint32_t*>(stage[warp]);
  auto value2 = [&](uint32_t h) {  // fp16 pair of codes -> bf16 pair of values
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_bf16x2(__fmul_rn(f.x, scale), __fmul_rn(f.y, scale));
  };
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    uint32_t y[4][4];
    if (kv) {
      const int idx = it * 32 + lane, t = idx / (HD / 8), c = idx % (HD / 8);
#pragma unroll
      for (int g = 0; g < 8; g += 2) {  // dims 8 c + g, + 1 of tokens 2t, 2t + 1, 2t + 8, 2t + 9
        uint32_t lo0, hi0, lo1, hi1;
        kv8_expand<FMT>(words[(c >> 2) * 128 + (g * 4 + t) * 4 + (c & 3)], lo0, hi0);
        kv8_expand<FMT>(words[(c >> 2) * 128 + (g * 4 + 4 + t) * 4 + (c & 3)], lo1, hi1);
        y[0][g >> 1] = value2(__byte_perm(lo0, lo1, 0x5410));
        y[1][g >> 1] = value2(__byte_perm(lo0, lo1, 0x7632));
        y[2][g >> 1] = value2(__byte_perm(hi0, hi1, 0x5410));
        y[3][g >> 1] = value2(__byte_perm(hi0, hi1, 0x7632));
      }
#pragma unroll
      for (int v = 0; v < 4; ++v)
        *reinterpret_cast<uint4*>(dst + (2 * t + (v & 1) + 8 * (v >> 1)) * HD + c * 8) =
            make_uint4(y[v][0], y[v][1], y[v][2], y[v][3]);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int idx = (2 * it + h) * 32 + lane, token = idx / (HD / 16), kk = idx % (HD / 16);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          uint32_t lo, hi;
          kv8_expand<FMT>(words[(kk >> 1) * 128 + ((token & 7) * 4 + t) * 4 + (kk & 1) * 2 + (token >> 3)], lo, hi);
          y[2 * h][t] = value2(lo);
          y[2 * h + 1][t] = value2(hi);
        }
        uint4* d = reinterpret_cast<uint4*>(dst + token * HD + kk * 16);
        d[0] = make_uint4(y[2 * h][0], y[2 * h][1], y[2 * h][2], y[2 * h][3]);
        d[1] = make_uint4(y[2 * h + 1][0], y[2 * h + 1][1], y[2 * h + 1][2], y[2 * h + 1][3]);
      }
    }
  }
}

// One block of 256 threads moves 16 KB of a page: four 16-byte words per thread,
// all loaded before the first is stored.
constexpr int kCopyBlock = 16384;
__global__ void __launch_bounds__(256) copy_pages_kernel(CopyArgs a, const __grid_constant__ PagePairs pairs, int parts) {
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

template <int HD>
int launch_seal_t(const SealArgs& a, const PagePairs& p, bool unseal, cudaStream_t s) {
  const long long units = static_cast<long long>(p.n) * a.layers * a.Hkv * 2;
  const dim3 grid(static_cast<unsigned>((units + 3) / 4));
  auto k = unseal ? (a.format == VD_KV8_INT8 ? kv8_unseal_kernel<HD, kKv8Int8> : kv8_unseal_kernel<HD, kKv8E4m3>)
                  : (a.format == VD_KV8_INT8 ? kv8_seal_kernel<HD, kKv8Int8> : kv8_seal_kernel<HD, kKv8E4m3>);
  VD_CUDA_TRY(launch_k(k, grid, dim3(128), 0, s, a, p));
  return VD_OK;
}

}  // namespace

int launch_kv8_seal(const SealArgs& a, const PagePairs& p, bool unseal, cudaStream_t s) {
  if (p.n <= 0) return VD_OK;
  if (a.hd == 64) return launch_seal_t<64>(a, p, unseal, s);
  if (a.hd == 128) return launch_seal_t<128>(a, p, unseal, s);
  if (a.hd == 256) return launch_seal_t<256>(a, p, unseal, s);
  return fail(VD_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
}

int launch_copy_pages(const CopyArgs& a, const PagePairs& p, cudaStream_t s) {
  if (p.n <= 0) return VD_OK;
  const int parts = static_cast<int>((a.bytes + kCopyBlock - 1) / kCopyBlock);
  VD_CUDA_TRY(launch_k(copy_pages_kernel, dim3(static_cast<unsigned>(p.n * a.layers * parts)), dim3(256), 0, s, a, p, parts));
  return VD_OK;
}

}  // namespace vd
