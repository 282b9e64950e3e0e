// Rotary positions for any pair layout, rotated part and frequency scaling.
//
// Pair i of a head turns by angle p * f_i at position p, f_i = theta^(-2i/rot)
// after scaling.  An angle is only needed modulo a full turn, so f_i / 2 pi
// is held as a 64-bit fraction of a turn, tau_i = floor(2^64 f_i / 2 pi), and
// p * tau_i in wrapping 64-bit integers *is* the reduced angle, where a float32
// product p * f_i would lose every bit of a far position's angle.  Its error is
// |p| times that of tau_i: 2^-64 turns for the floor, and as much again for f_i,
// which is made in long double (64 bits or more) and at most 1 unless a scaling
// factor below 1 makes it larger: 2^-32 turns at the largest int32 position (a
// frequency held as a double would be off by 2^-25 there).  The two top bits
// (after rounding to the nearest quarter) are the quadrant, the rest is rounded
// to a float32 in [-1/4, 1/4] half-turns, by 2^-28 turns at most, for sincospif.
// No table is read: a handle works for every position, on every device and
// stream.
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>
#include <new>

#include "vd_device.cuh"
#include "vd_internal.h"
#include "vd_model.h"

using namespace vd;

namespace vd {

// The frequencies, by value in the kernel's parameters (2 KB).
struct RopeTurns {
  unsigned long long turn[kRopeMaxPairs];
};

}  // namespace vd

struct vd_rope {
  vd_rope_config cfg{};
  int rot = 0;
  float mag = 1.f;      // magnitude of the rotation (YaRN's attention factor)
  float inv_mag = 1.f;
  RopeTurns turns{};
};

namespace {

// cos and sin of position p's angle, times mag.
__device__ __forceinline__ float2 turn_cs(unsigned long long tau, int p, float mag) {
  const unsigned long long a = tau * static_cast<unsigned long long>(static_cast<long long>(p));
  const unsigned q = static_cast<unsigned>((a + (1ull << 61)) >> 62);  // nearest quarter turn
  const long long r = static_cast<long long>(a - (static_cast<unsigned long long>(q) << 62));
  float s, c;
  sincospif(__fmul_rn(static_cast<float>(r), 1.0842021724855044e-19f), &s, &c);  // r * 2^-63 half-turns
  const float cr = q & 1 ? s : c, sr = q & 1 ? c : s;  // swap on odd quarters, then signs
  return make_float2(__fmul_rn(q == 1 || q == 2 ? -cr : cr, mag), __fmul_rn(q >= 2 ? -sr : sr, mag));
}

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(float x) { return x; }
template <>
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }

struct RotaryArgs {
  const void* x;
  void* y;
  const int* pos;
  long long xs_t, xs_h, ys_t, ys_h;  // strides in elements
  int T, H, hd, rot;
  int rest;      // 1: copy dims [rot, hd) (0 when rotating in place)
  int inverse;
  float mag;
};

// E consecutive elements, one 16-byte access for E > 1.
template <typename T, int E>
struct Pack {
  T v[E];
};
template <typename T, int E>
__device__ __forceinline__ Pack<T, E> load_pack(const T* p) {
  Pack<T, E> r;
  if constexpr (E > 1) {
    static_assert(sizeof(T) * E == 16, "16-byte packs");
    *reinterpret_cast<uint4*>(&r) = *reinterpret_cast<const uint4*>(p);
  } else {
    r.v[0] = *p;
  }
  return r;
}
template <typename T, int E>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, E>& r) {
  if constexpr (E > 1)
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(&r);
  else
    *p = r.v[0];
}

// Block (x: a head's chunks, y: heads, z: tokens).  A chunk is two packs: half
// layout, elements i.. of the first half and of the second; interleaved, 2E
// neighbours.  A thread's first kUnroll heads are loaded before anything else,
// so that the position's round trip, the cosines and sines (once per token for
// all heads) and the barrier pass while the data is on its way.
// Bound by memory: 8192 tokens x 40 heads x 128 dims of bf16 in rows of 48 heads
// move 168 MB in 30.9 us (5.4 TB/s, 0.80 of the copy peak; heads one after the
// other, loaded behind the barrier, took 64 us); 4097 x 13 x 96 float32 with 64
// dims rotated, 41 MB in 9.6 us.  64 tokens take 4.3 us, less than their launch
// from Python (6 us).
constexpr int kUnroll = 4;
template <typename T, int E, bool INTER>
__global__ void __launch_bounds__(256) rotary_kernel(const __grid_constant__ RopeTurns turns, RotaryArgs a) {
  extern __shared__ float cs_s[];  // [tokens][2][pairs]: cosines, then sines
  const int pairs = a.rot >> 1, chunks = pairs / E;
  const int total = chunks + (a.rest ? (a.hd - a.rot) / (2 * E) : 0);
  const int tid = threadIdx.x + blockDim.x * (threadIdx.y + blockDim.y * threadIdx.z);
  const int threads = blockDim.x * blockDim.y * blockDim.z;
  const long long t0 = static_cast<long long>(blockIdx.x) * blockDim.z;
  const int nt = static_cast<int>(min(static_cast<long long>(blockDim.z), a.T - t0));
  const int tt = threadIdx.z;
  const T* x = static_cast<const T*>(a.x) + (t0 + tt) * a.xs_t;
  T* y = static_cast<T*>(a.y) + (t0 + tt) * a.ys_t;
  int ch = threadIdx.x, h0 = threadIdx.y;
  Pack<T, E> p0[kUnroll], p1[kUnroll];
  auto offsets = [&](int& o0, int& o1) {  // the chunk's two packs
    const bool split = ch < chunks && !INTER;
    o0 = split ? ch * E : ch * 2 * E;
    o1 = split ? o0 + pairs : o0 + E;
  };
  auto load = [&] {
    int o0, o1;
    offsets(o0, o1);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * blockDim.y;
      if (h >= a.H) continue;
      p0[u] = load_pack<T, E>(x + h * a.xs_h + o0);
      p1[u] = load_pack<T, E>(x + h * a.xs_h + o1);
    }
  };
  pdl_wait();
  pdl_trigger();
  if (tt < nt && ch < total) load();
  for (int k = tid; k < nt * pairs; k += threads) {
    const int tk = k / pairs, i = k % pairs;
    const float2 c = turn_cs(turns.turn[i], a.pos[t0 + tk], a.mag);
    cs_s[(2 * tk) * pairs + i] = c.x;
    cs_s[(2 * tk + 1) * pairs + i] = a.inverse ? -c.y : c.y;
  }
  __syncthreads();
  if (tt >= nt) return;
  bool loaded = true;
  for (; ch < total; ch += blockDim.x) {
    const bool rot = ch < chunks;
    float c[E], s[E];
    if (rot) {
#pragma unroll
      for (int k = 0; k < E; ++k) {
        c[k] = cs_s[(2 * tt) * pairs + ch * E + k];
        s[k] = cs_s[(2 * tt + 1) * pairs + ch * E + k];
      }
    }
    int o0, o1;
    offsets(o0, o1);
    for (h0 = threadIdx.y; h0 < a.H; h0 += blockDim.y * kUnroll) {
      if (!loaded) load();
      loaded = false;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = h0 + u * blockDim.y;
        if (h >= a.H) continue;
        if (rot) {
#pragma unroll
          for (int k = 0; k < E; ++k) {
            // pair k of the chunk: (p0[k], p1[k]), or neighbours 2k, 2k + 1 of the two packs
            T& r1 = !INTER ? p0[u].v[k] : 2 * k < E ? p0[u].v[(2 * k) % E] : p1[u].v[(2 * k) % E];
            T& r2 = !INTER ? p1[u].v[k] : 2 * k + 1 < E ? p0[u].v[(2 * k + 1) % E] : p1[u].v[(2 * k + 1) % E];
            const float x1 = to_f(r1), x2 = to_f(r2);
            r1 = from_f<T>(__fsub_rn(__fmul_rn(x1, c[k]), __fmul_rn(x2, s[k])));
            r2 = from_f<T>(__fadd_rn(__fmul_rn(x2, c[k]), __fmul_rn(x1, s[k])));
          }
        }
        store_pack<T, E>(y + h * a.ys_h + o0, p0[u]);
        store_pack<T, E>(y + h * a.ys_h + o1, p1[u]);
      }
    }
  }
}

// Rotation tables of a model: cos, sin [positions][half], mag included;
// entries past the rotated pairs are not read.
__global__ void rope_table_kernel(const __grid_constant__ RopeTurns turns, int positions, int pairs, int half, float mag,
                                  float* cs, float* sn) {
  const long long k = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (k >= static_cast<long long>(positions) * pairs) return;
  const int p = static_cast<int>(k / pairs), i = static_cast<int>(k % pairs);
  const float2 c = turn_cs(turns.turn[i], p, mag);
  cs[static_cast<size_t>(p) * half + i] = c.x;
  sn[static_cast<size_t>(p) * half + i] = c.y;
}

template <typename T, int E>
int launch_rotary(const vd_rope* r, const RotaryArgs& a, cudaStream_t s) {
  const int pairs = a.rot / 2;
  const int total = pairs / E + (a.rest ? (a.hd - a.rot) / (2 * E) : 0);
  // up to 256 threads: the chunks of a head, every kUnroll-th head, then tokens
  dim3 block(std::min(total, 128), 1, 1);
  block.y = std::max(1, std::min<int>((a.H + kUnroll - 1) / kUnroll, 256 / block.x));
  block.z = std::max(1, std::min<int>({a.T, 8, static_cast<int>(256 / (block.x * block.y))}));
  const unsigned blocks = (static_cast<unsigned>(a.T) + block.z - 1) / block.z;
  const size_t smem = static_cast<size_t>(block.z) * a.rot * sizeof(float);
  auto k = r->cfg.layout == VD_ROPE_INTERLEAVED ? rotary_kernel<T, E, true> : rotary_kernel<T, E, false>;
  VD_CUDA_TRY(launch_k(k, dim3(blocks), block, smem, s, r->turns, a));
  return VD_OK;
}

template <typename T>
int launch_rotary_t(const vd_rope* r, const RotaryArgs& a, cudaStream_t s) {
  constexpr int E = 16 / sizeof(T);
  // 16-byte packs where every pack starts on a 16-byte boundary, else element by element
  const bool packed = aligned16(a.x) && aligned16(a.y) && a.xs_t % E == 0 && a.xs_h % E == 0 && a.ys_t % E == 0 &&
                      a.ys_h % E == 0 && a.rot % (2 * E) == 0 && (!a.rest || (a.hd - a.rot) % (2 * E) == 0);
  return packed ? launch_rotary<T, E>(r, a, s) : launch_rotary<T, 1>(r, a, s);
}

bool bad(double v) { return !(v > 0) || isinf(v); }

// Whether two of the rows [t * st + h * sh, + hd), t < T and h < H, share an
// element: |dt * st + dh * sh| < hd for some differences, not both zero.
bool rows_overlap(int T, int H, long long st, long long sh, int hd) {
  using wide = __int128;
  const wide at = st < 0 ? -wide(st) : wide(st), ah = sh < 0 ? -wide(sh) : wide(sh);
  if ((T > 1 && at < hd) || (H > 1 && ah < hd)) return true;
  if (T == 1 || H == 1) return false;
  // rows of the smaller stride, again after every larger one: nested, or interleaved and looked at one by one
  const wide small = at < ah ? at : ah, large = at < ah ? ah : at;
  const wide n_small = at < ah ? T : H, n_large = at < ah ? H : T, span = (n_small - 1) * small;
  for (wide d = 1; d < n_large && d * large < span + hd; ++d) {
    const wide below = d * large / small, rest = d * large % small;
    if ((below < n_small && rest < hd) || (below + 1 < n_small && small - rest < hd)) return true;
  }
  return false;
}

}  // namespace

extern "C" {

int vd_rope_create(const vd_rope_config* cfg, vd_rope** out) {
  if (!cfg || !out) return fail(VD_ERR_INVALID_ARG, "null argument");
  *out = nullptr;
  const vd_rope_config& c = *cfg;
  const int rot = c.rot_dim == 0 ? c.head_dim : c.rot_dim;
  if (c.head_dim < 2 || c.head_dim % 2 || rot < 2 || rot % 2 || rot > c.head_dim)
    return fail(VD_ERR_INVALID_ARG, "head_dim and rot_dim must be even, 2 <= rot_dim <= head_dim");
  if (rot / 2 > kRopeMaxPairs) return fail(VD_ERR_UNSUPPORTED, "at most 512 rotated dims");
  if (c.layout != VD_ROPE_HALF && c.layout != VD_ROPE_INTERLEAVED) return fail(VD_ERR_INVALID_ARG, "unknown layout");
  if (!(c.theta > 1) || isinf(c.theta)) return fail(VD_ERR_INVALID_ARG, "theta must be above 1");
  if (c.scaling < VD_ROPE_SCALE_NONE || c.scaling > VD_ROPE_SCALE_YARN)
    return fail(VD_ERR_INVALID_ARG, "unknown scaling");
  if (c.scaling != VD_ROPE_SCALE_NONE && bad(c.factor)) return fail(VD_ERR_INVALID_ARG, "factor must be positive");
  if (c.scaling == VD_ROPE_SCALE_BANDS &&
      (bad(c.low_freq_factor) || bad(c.high_freq_factor) || c.high_freq_factor <= c.low_freq_factor ||
       bad(c.original_max_position)))
    return fail(VD_ERR_INVALID_ARG, "bands need 0 < low_freq_factor < high_freq_factor and original_max_position > 0");
  if (c.scaling == VD_ROPE_SCALE_YARN &&
      (bad(c.beta_fast) || bad(c.beta_slow) || c.beta_fast <= c.beta_slow || bad(c.original_max_position)))
    return fail(VD_ERR_INVALID_ARG, "YaRN needs 0 < beta_slow < beta_fast and original_max_position > 0");
  if (!(c.attn_factor >= 0) || isinf(c.attn_factor)) return fail(VD_ERR_INVALID_ARG, "attn_factor must be >= 0");
  const double two_pi = 6.283185307179586476925286766559;
  double ylo = 0, yhi = 0, mag = c.attn_factor > 0 ? c.attn_factor : 1.0;
  if (c.scaling == VD_ROPE_SCALE_YARN) {
    auto dim_of = [&](double turns) {  // the pair that turns this often within the original context
      return rot * log(c.original_max_position / (turns * two_pi)) / (2.0 * log(c.theta));
    };
    ylo = std::max(floor(dim_of(c.beta_fast)), 0.0);
    yhi = std::min(ceil(dim_of(c.beta_slow)), rot - 1.0);
    if (c.attn_factor == 0 && c.factor > 1) mag = 0.1 * log(c.factor) + 1.0;
  }
  if (!isnormal(static_cast<float>(mag)) || !isnormal(static_cast<float>(1.0 / mag)))
    return fail(VD_ERR_INVALID_ARG, "attn_factor and its inverse must be float32 numbers");
  vd_rope* r = new (std::nothrow) vd_rope();
  if (!r) return fail(VD_ERR_CAPACITY, "out of host memory");
  r->cfg = c;
  r->rot = rot;
  r->mag = static_cast<float>(mag);
  r->inv_mag = static_cast<float>(1.0 / mag);
  // in extended precision: a position of 2^31 multiplies what a double leaves off
  using real = long double;
  const real full = 6.283185307179586476925286766559005768L;
  for (int i = 0; i < rot / 2; ++i) {
    real f = powl(c.theta, -2.0L * i / rot);
    if (c.scaling == VD_ROPE_SCALE_LINEAR) f /= c.factor;
    if (c.scaling == VD_ROPE_SCALE_BANDS) {
      const real turns = c.original_max_position * f / full;
      const real keep = (turns - c.low_freq_factor) / (static_cast<real>(c.high_freq_factor) - c.low_freq_factor);
      const real k = std::min(std::max(keep, 0.0L), 1.0L);
      f = k * f + (1 - k) * f / c.factor;
    }
    if (c.scaling == VD_ROPE_SCALE_YARN) {
      const real ramp = std::min(std::max((i - ylo) / (yhi > ylo ? yhi - ylo : static_cast<real>(0.001)), 0.0L), 1.0L);
      f = (1 - ramp) * f + ramp * f / c.factor;
    }
    // turns per position in units of 2^-64; whole turns (factors below 1) drop out
    const real turns = f / full, frac = turns - floorl(turns);
    r->turns.turn[i] = static_cast<unsigned long long>(ldexpl(frac, 64));
  }
  *out = r;
  return VD_OK;
}

void vd_destroy_rope(vd_rope* r) { delete r; }

int vd_op_rotary(const vd_rope* r, const void* x, void* y, int32_t T, int32_t H, int64_t x_stride_t, int64_t x_stride_h,
                 int64_t y_stride_t, int64_t y_stride_h, int32_t dtype, const int32_t* positions, int32_t inverse,
                 void* stream) {
  if (!r) return fail(VD_ERR_INVALID_ARG, "null rope");
  if (T < 0 || H < 0) return fail(VD_ERR_INVALID_ARG, "negative size");
  if (dtype < VD_DTYPE_BF16 || dtype > VD_DTYPE_F32) return fail(VD_ERR_INVALID_ARG, "unknown dtype");
  if (inverse != 0 && inverse != 1) return fail(VD_ERR_INVALID_ARG, "inverse must be 0 or 1");
  if (T == 0 || H == 0) return VD_OK;
  if (!x || !y || !positions) return fail(VD_ERR_INVALID_ARG, "null pointer");
  const int size = dtype == VD_DTYPE_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) % size ||
      reinterpret_cast<uintptr_t>(positions) % 4)
    return fail(VD_ERR_INVALID_ARG, "pointer not aligned to its type");
  const int hd = r->cfg.head_dim;
  // the rows y[t][h] must not overlap one another, nor x's (but for the same rows in place)
  if (rows_overlap(T, H, y_stride_t, y_stride_h, hd))
    return fail(VD_ERR_INVALID_ARG, "rows of y overlap");
  const bool in_place = x == y;
  if (in_place && ((T > 1 && x_stride_t != y_stride_t) || (H > 1 && x_stride_h != y_stride_h)))
    return fail(VD_ERR_INVALID_ARG, "in place, the strides of x and y must be equal");
  RotaryArgs a{};
  a.x = x;
  a.y = y;
  a.pos = positions;
  a.xs_t = T > 1 ? x_stride_t : 0;
  a.xs_h = H > 1 ? x_stride_h : 0;
  a.ys_t = T > 1 ? y_stride_t : 0;
  a.ys_h = H > 1 ? y_stride_h : 0;
  a.T = T;
  a.H = H;
  a.hd = hd;
  a.rot = r->rot;
  a.rest = !in_place && r->rot < hd;
  a.inverse = inverse;
  a.mag = inverse ? r->inv_mag : r->mag;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == VD_DTYPE_F32) return launch_rotary_t<float>(r, a, s);
  if (dtype == VD_DTYPE_F16) return launch_rotary_t<__half>(r, a, s);
  return launch_rotary_t<__nv_bfloat16>(r, a, s);
}

int vd_set_rope(vd_model* m, const vd_rope* global, const vd_rope* local) {
  if (check_model(m)) return VD_ERR_INVALID_ARG;
  if (!global) return fail(VD_ERR_INVALID_ARG, "null rope");
  if (!local) local = global;
  const int hd = m->cfg.head_dim;
  if (global->cfg.head_dim != hd || local->cfg.head_dim != hd)
    return fail(VD_ERR_INVALID_ARG, "the ropes' head_dim differs from the model's");
  int dev = -1;
  VD_CUDA_TRY(cudaGetDevice(&dev));
  if (dev != m->device) return fail(VD_ERR_INVALID_ARG, "the model lives on another device than the current one");
  // steps in flight and captured graphs read the tables: wait for the first, drop the second
  VD_CUDA_TRY(cudaDeviceSynchronize());
  drop_graphs(m);
  const struct {
    const vd_rope* r;
    float *cs, *sn;
    RopeShape* shape;
  } set[2] = {{global, m->cos_g, m->sin_g, &m->rope_g}, {local, m->cos_l, m->sin_l, &m->rope_l}};
  for (const auto& x : set) {
    const int pairs = x.r->rot / 2;
    const long long n = static_cast<long long>(m->cfg.max_context) * pairs;
    rope_table_kernel<<<static_cast<unsigned>((n + 255) / 256), 256>>>(x.r->turns, m->cfg.max_context, pairs, hd / 2,
                                                                      x.r->mag, x.cs, x.sn);
    VD_CUDA_TRY(cudaGetLastError());
    x.shape->rot = x.r->rot == hd ? 0 : x.r->rot;
    x.shape->interleaved = x.r->cfg.layout == VD_ROPE_INTERLEAVED;
  }
  VD_CUDA_TRY(cudaDeviceSynchronize());
  return VD_OK;
}

}  // extern "C"
