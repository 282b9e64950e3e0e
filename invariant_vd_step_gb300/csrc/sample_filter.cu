// Token choice with temperature, top-k, top-p and min-p.
//
// A row's kept tokens are a prefix of its tokens in descending order (ties:
// lower index first), cut by the filters that are on: the top_k first; those
// before which the probability mass is below top_p; those whose probability is
// at least min_p of the largest.  The choice is the Gumbel-max choice of
// sampler.cu over the kept tokens, with the same random numbers and the same
// scores, so that a row without filters gets exactly vd_sample's token.
//
// Almost every row is decided by a few dozen of its V logits.  Pass 1 reads
// the logits once, at memory speed: a warp takes a segment of 1024, finds its
// maximum, its sum of exponentials and a threshold that at least `keep` of
// its logits reach (the keep-th largest of the 32 lanes' maxima), and writes
// the logits from that threshold on to a short list.  Every logit at or above
// the largest threshold of a row's segments is then in a list.  Pass 2, one
// cluster per row, sorts as many listed candidates as it needs and walks down
// them.  Where the cut lies below the lists (flat distributions, huge top_k,
// logits sorted by value along the vocabulary), the cluster re-reads the row:
// a histogram over 2048 bins of value finds the bin of the cut, bins of the
// (value, index) order refine it until it holds at most kList tokens, and one
// more pass scores everything above the bin and collects it.
//
// Sums that decide something do not depend on timing: candidate masses are
// summed in sorted order, histogram masses as 64-bit integers.
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "vd_device.cuh"
#include "vd_internal.h"

namespace vd {
namespace {

constexpr int kSeg = 1024;        // logits of a segment (one warp: 8 x 4 per lane)
constexpr int kSegCap = 64;       // list entries per segment
constexpr int kScanThreads = 256;
constexpr int kSelThreads = 256;
constexpr int kBins = 2048;
constexpr int kList = 2048;       // candidates that pass 2 sorts
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMassScale = 68719476736.f;  // 2^36: fixed-point unit of histogram masses (V <= 2^21: sums below 2^57)

enum RowMode { ROW_GREEDY = 0, ROW_FREE = 1, ROW_FILTER = 2 };

struct RowParam {
  uint64_t seed, step;
  float temp, top_p, log_min_p;  // top_p >= 1: off; log_min_p = -inf: off
  int top_k;                     // 0: off
};
template <int N>
struct RowParams {
  RowParam r[N];
};
__device__ __forceinline__ int row_mode(const RowParam& p) {
  if (!(p.temp > 0.f)) return ROW_GREEDY;
  return p.top_k > 0 || p.top_p < 1.f || p.log_min_p > -INFINITY ? ROW_FILTER : ROW_FREE;
}

// What pass 1 leaves of a segment.
struct __align__(32) SegOut {
  float max, sum;   // largest logit; sum of exp((l - max) / T)
  uint32_t thr;     // every logit whose key is at least this is in the list
  int count;        // list entries
  float best;       // greedy and unfiltered rows: the best score
  int best_i;
  int pad_[2];
};

// Order of the logits: NaN lowest (key 0, never chosen), then by value with
// -0 = +0; `comp` adds the index, lower first.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t u = __float_as_uint(__fadd_rn(l, 0.f));
  return l != l ? 0u : u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key >> 31 ? key ^ 0x80000000u : ~key);
}
constexpr uint32_t kKeyLowest = 0x00800000u;  // of the lowest finite value; -inf is below it
__device__ __forceinline__ uint64_t comp_of(float l, int i) {
  return (static_cast<uint64_t>(key_of(l)) << 32) | static_cast<uint32_t>(~i);
}
__device__ __forceinline__ int index_of(uint64_t comp) { return static_cast<int>(~static_cast<uint32_t>(comp)); }

// exp((l - m) / T) for l <= m, c = log2(e) / T; 1 at m itself (also for m
// infinite), 0 for NaN.
__device__ __forceinline__ float weight(float l, float m, float c) {
  const float w = ex2(__fmul_rn(__fsub_rn(l, m), c));
  return l == m ? 1.f : w == w ? w : 0.f;
}

// The best Gumbel score of a stream of tokens, without the two logarithms
// for tokens that cannot win: G = -log(-log u) <= -log(1 - u), so a token
// beats `best` only if 1 - u <= exp(x - best).  The test errs on the side of
// scoring (1e-3 and 2^-21 of the magnitudes cover its own rounding and that of
// the score), so the winner is the one that scoring every token finds.
struct Race {
  float best = -INFINITY;
  int best_i = INT_MAX;
  float lim = -INFINITY;  // best less its margin
  __device__ __forceinline__ void set_lim() {
    lim = __fsub_rn(best, __fadd_rn(__fmul_rn(fabsf(best), 4.76837158203125e-7f), 1e-3f));
  }
  __device__ __forceinline__ void take(float v, int i) {
    if (better(v, i, best, best_i)) {
      best = v;
      best_i = i;
      set_lim();
    }
  }
  // inv_t = 1 / T
  __device__ __forceinline__ void token(float l, int i, uint32_t word, float t, float inv_t) {
    const float x = __fmul_rn(l, inv_t);
    const float rest = __fmul_rn(__fadd_rn(static_cast<float>(0xFFFFFFu - (word >> 8)), 0.5f), 5.9604644775390625e-8f);
    const float a = ex2(__fmul_rn(__fsub_rn(__fadd_rn(x, __fmul_rn(fabsf(x), 4.76837158203125e-7f)), lim), kLog2e));
    if (!(rest > a)) take(gumbel_score(l, word, t), i);
  }
  // over the warp; every lane ends with the winner
  __device__ __forceinline__ void warp_reduce() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float ov = __shfl_xor_sync(0xffffffffu, best, o);
      const int oi = __shfl_xor_sync(0xffffffffu, best_i, o);
      if (better(ov, oi, best, best_i)) {
        best = ov;
        best_i = oi;
      }
    }
    set_lim();
  }
};

__device__ __forceinline__ uint32_t word_of(const uint4& w, int e) {
  return e == 0 ? w.x : e == 1 ? w.y : e == 2 ? w.z : w.w;
}

// The four logits from index i0 (a multiple of 4); NaN past the row's end.
template <bool VEC>
__device__ __forceinline__ float4 load4(const float* row, int i0, int V) {
  if (VEC && i0 + 4 <= V) return *reinterpret_cast<const float4*>(row + i0);
  float4 v = make_float4(NAN, NAN, NAN, NAN);
  if (i0 < V) v.x = row[i0];
  if (i0 + 1 < V) v.y = row[i0 + 1];
  if (i0 + 2 < V) v.z = row[i0 + 2];
  if (i0 + 3 < V) v.w = row[i0 + 3];
  return v;
}

// ---------------------------------------------------------------- pass 1
template <int N, bool VEC>
__global__ void __launch_bounds__(kScanThreads)
    filter_scan_kernel(const __grid_constant__ RowParams<N> params, const float* __restrict__ logits, int V,
                       long long ld, int nseg, int keep, SegOut* __restrict__ segs, uint64_t* __restrict__ lists) {
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seg = blockIdx.x * (kScanThreads / 32) + warp;
  if (seg >= nseg) return;
  const float* row = logits + r * ld;
  const int i0 = seg * kSeg + lane * 4;
  float v[8][4];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float4 x = load4<VEC>(row, i0 + q * 128, V);
    v[q][0] = x.x;
    v[q][1] = x.y;
    v[q][2] = x.z;
    v[q][3] = x.w;
  }
  const RowParam p = params.r[r];
  const int mode = row_mode(p);
  float lm = -INFINITY;
#pragma unroll
  for (int q = 0; q < 8; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) lm = fmaxf(lm, v[q][e]);
  float m = lm;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  SegOut out{};
  out.max = m;
  Race race;
  if (mode == ROW_GREEDY || m == -INFINITY) {
    // the lowest index among the maxima; a row of NaN and -inf has its lowest -inf
#pragma unroll
    for (int q = 7; q >= 0; --q)
#pragma unroll
      for (int e = 3; e >= 0; --e)
        if (v[q][e] == m) race.best_i = i0 + q * 128 + e;
    race.best = race.best_i == INT_MAX ? -INFINITY : m;
    race.warp_reduce();
  } else {
    const float c = __fdiv_rn(kLog2e, p.temp);
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum = __fadd_rn(sum, weight(v[q][e], m, c));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
    out.sum = sum;
    if (mode == ROW_FREE) {
      const float inv_t = __fdiv_rn(1.f, p.temp);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int i = i0 + q * 128;
        const uint4 w = philox_block(p.seed, p.step, static_cast<uint32_t>(i) / 4);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e < V) race.token(v[q][e], i + e, word_of(w, e), p.temp, inv_t);
        if (q == 0) race.warp_reduce();  // a bound for the rest of the segment
      }
      race.warp_reduce();
    } else {
      // lane maxima in descending order (bitonic, over the warp)
      float s = lm;
#pragma unroll
      for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
          const float o = __shfl_xor_sync(0xffffffffu, s, j);
          const bool up = ((lane & k) == 0) == ((lane & j) == 0);  // this lane keeps the larger
          s = up ? fmaxf(s, o) : fminf(s, o);
        }
      // the lowest threshold whose list fits: the keep-th lane maximum, else a higher one, else none
      out.thr = key_of(m) + 1;
      uint64_t* list = lists + (static_cast<size_t>(r) * nseg + seg) * kSegCap;
      for (int rank = keep - 1; rank >= 0; rank = rank > 3 ? 3 : rank > 0 ? 0 : -1) {
        const uint32_t t = max(key_of(__shfl_sync(0xffffffffu, s, rank)), kKeyLowest);  // -inf is never listed
        const float tv = value_of(t);
        int n = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) n += v[q][e] >= tv;
        int before = n;  // inclusive prefix sum over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += x;
        }
        const int total = __shfl_sync(0xffffffffu, before, 31);
        if (total > kSegCap) continue;
        before -= n;
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (v[q][e] >= tv) list[before++] = comp_of(v[q][e], i0 + q * 128 + e);
        out.thr = t;
        out.count = total;
        break;
      }
    }
  }
  out.best = race.best;
  out.best_i = race.best_i;
  if (out.thr == 0) out.thr = kKeyLowest;  // nothing to list
  if (lane == 0) segs[static_cast<size_t>(r) * nseg + seg] = out;
}

// ---------------------------------------------------------------- pass 2
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address, in the cluster's shared window, of CTA `rank`'s copy of p.
__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t peer_ld32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t peer_ld64(uint32_t a) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void peer_st32(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void peer_st64(uint32_t a, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t peer_add32(uint32_t a, uint32_t v) {
  uint32_t o;
  asm volatile("atom.add.shared::cluster.u32 %0, [%1], %2;" : "=r"(o) : "r"(a), "r"(v) : "memory");
  return o;
}

// Shared memory of a CTA.  The histogram and the sorted list are never in use
// at the same time.
struct SelShared {
  union {
    struct {
      uint32_t cnt[kBins], lo[kBins], hi[kBins];  // tokens; masses as 64-bit integers in two words
    } h;
    struct {
      uint64_t comp[kList];
      double pre[kList];  // masses up to and including each
    } l;
  };
  double redd[kSelThreads / 32];
  float redf[kSelThreads / 32];
  int redi[kSelThreads / 32];
  uint64_t redu[kSelThreads / 32];
  int go;                    // the row has to be re-read
  float top;                 // its largest logit
  int n;                     // list entries
  uint64_t clo, chi;         // tokens of the undecided bin (comp range, inclusive)
  uint64_t above_mass;       // of the tokens above it
  uint32_t above_cnt, in_cnt;
  uint64_t last_comp;        // the top_k-th token, where top-p cuts within top-k
  uint64_t total_mass;
  float r_best[16];          // per rank: the best of the tokens above the bin
  int r_best_i[16];
  uint64_t r_mass[16];
};

template <typename T, typename Op>
__device__ __forceinline__ T block_reduce(T v, T* red, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();  // red's earlier readers are done
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < kSelThreads / 32; ++w) v = op(v, red[w]);
  return v;
}

// Sorts comp[0, n) in descending order (n <= kList, the values all different).
__device__ void sort_desc(uint64_t* comp, int n) {
  if (n <= kSelThreads) {  // by rank: each thread counts the values above its own
    const int i = threadIdx.x;
    const uint64_t mine = i < n ? comp[i] : 0;
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += comp[j] > mine;
    __syncthreads();
    if (i < n) comp[rank] = mine;
    __syncthreads();
    return;
  }
  int p = 2 * kSelThreads;
  while (p < n) p <<= 1;
  for (int i = n + threadIdx.x; i < p; i += kSelThreads) comp[i] = 0;
  __syncthreads();
  for (int k = 2; k <= p; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int t = threadIdx.x; t < p / 2; t += kSelThreads) {
        const int a = 2 * t - (t & (j - 1)), b = a + j;
        const uint64_t x = comp[a], y = comp[b];
        if ((x < y) == ((a & k) == 0)) {
          comp[a] = y;
          comp[b] = x;
        }
      }
      __syncthreads();
    }
}

// pre[j] = base + weights of comp[0 .. j], summed in that order.
__device__ void prefix_mass(SelShared& sh, int n, float top, float t, double base) {
  const int per = (n + kSelThreads - 1) / kSelThreads, j0 = threadIdx.x * per;
  double sum = 0;
  for (int j = j0; j < min(n, j0 + per); ++j) {
    const float l = value_of(static_cast<uint32_t>(sh.l.comp[j] >> 32));
    sum += l == top ? 1.0 : static_cast<double>(expf(__fdiv_rn(__fsub_rn(l, top), t)));
    sh.l.pre[j] = sum;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double s = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double x = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += x;
  }
  __syncthreads();
  if (lane == 31) sh.redd[warp] = s;
  __syncthreads();
  double off = base + (s - sum);
  for (int w = 0; w < warp; ++w) off += sh.redd[w];
  for (int j = j0; j < min(n, j0 + per); ++j) sh.l.pre[j] += off;
  __syncthreads();
}

__device__ __forceinline__ bool min_p_keeps(float l, float top, float t, float log_min_p) {
  return l == top || __fdiv_rn(__fsub_rn(l, top), t) >= log_min_p;
}

// The choice among the first `kept` of the sorted list and `race` (the best
// of tokens outside it); mass: that of every kept token.
__device__ void choose(SelShared& sh, const RowParam& p, int kept, Race race, double mass, float top, const float* row,
                       int* token_out, float* logprob_out) {
  for (int j = threadIdx.x; j < kept; j += kSelThreads) {
    const uint64_t cp = sh.l.comp[j];
    const int i = index_of(cp);
    const uint4 w = philox_block(p.seed, p.step, static_cast<uint32_t>(i) / 4);
    const float v = gumbel_score(value_of(static_cast<uint32_t>(cp >> 32)), word_of(w, i & 3), p.temp);
    if (better(v, i, race.best, race.best_i)) {
      race.best = v;
      race.best_i = i;
    }
  }
  race.warp_reduce();
  const int warp = threadIdx.x >> 5;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    sh.redf[warp] = race.best;
    sh.redi[warp] = race.best_i;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kSelThreads / 32; ++w)
      if (better(sh.redf[w], sh.redi[w], race.best, race.best_i)) {
        race.best = sh.redf[w];
        race.best_i = sh.redi[w];
      }
    const int tok = race.best_i == INT_MAX ? 0 : race.best_i;
    *token_out = tok;
    if (logprob_out) {
      const float l = row[tok];
      const float d = l == top ? 0.f : __fdiv_rn(__fsub_rn(l, top), p.temp);
      *logprob_out = __fsub_rn(d, log1pf(static_cast<float>(mass - 1.0)));
    }
  }
}

struct SelectArgs {
  const float* logits;
  long long ld;
  int V, nseg;
  const SegOut* segs;
  const uint64_t* lists;
  int* tokens;
  float* logprobs;  // or null
};

// The cluster's re-read of a row: f(four logits, their index / 4) over this
// CTA's part.
template <bool VEC, typename F>
__device__ __forceinline__ void for_slice(const float* row, int V, uint32_t rank, uint32_t size, F f) {
  const int quads = (V + 3) / 4, per = (quads + size - 1) / size;
  const int q0 = rank * per, q1 = min(quads, q0 + per);
  for (int q = q0 + threadIdx.x; q < q1; q += 4 * kSelThreads) {
    float4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (q + u * kSelThreads < q1) x[u] = load4<VEC>(row, (q + u * kSelThreads) * 4, V);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (q + u * kSelThreads < q1) f(x[u], q + u * kSelThreads);
  }
}

// Bin of a token: by value below `top` at first (the last bin takes
// everything further down), then by its place in [clo, chi].
struct Binner {
  bool first;
  float top, scale;    // first: bins per unit of (top - l)
  uint64_t clo, chi;
  int shift;
  __device__ __forceinline__ int operator()(float l, uint64_t comp) const {
    if (first) {
      const float d = l == top ? 0.f : __fmul_rn(__fsub_rn(top, l), scale);
      return d < static_cast<float>(kBins - 1) ? static_cast<int>(d) : kBins - 1;
    }
    return static_cast<int>((chi - comp) >> shift);
  }
};

// One histogram over the tokens of [clo, chi] (and, on the first pass, the
// universe comp >= ulo), merged over the cluster; then the bin where the
// criterion cuts.  by_count: the bin of the target-th token, else the bin in
// which the mass before a token reaches `share` of the total.  Narrows
// sh.clo / chi and adds to above_mass / above_cnt on every rank.
template <bool VEC>
__device__ void histogram_cut(SelShared& sh, const float* row, int V, const RowParam& p, bool first, uint64_t ulo,
                              bool by_count, int target, float share) {
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const float c = __fdiv_rn(kLog2e, p.temp), top = sh.top;
  Binner bin;
  bin.first = first;
  bin.top = top;
  bin.scale = __fdiv_rn(static_cast<float>(kBins) / 24.f, p.temp);  // 24 nats over the bins
  bin.clo = sh.clo;
  bin.chi = sh.chi;
  bin.shift = max(0, 64 - __clzll(static_cast<long long>(sh.chi - sh.clo)) - 11);
  const uint64_t clo = max(sh.clo, ulo), chi = sh.chi;
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kSelThreads) sh.h.cnt[i] = sh.h.lo[i] = sh.h.hi[i] = 0;
  __syncthreads();
  for_slice<VEC>(row, V, rank, size, [&](const float4& x, int q) {
    const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint64_t cp = comp_of(v[e], q * 4 + e);
      if (cp < clo || cp > chi) continue;
      const int b = bin(v[e], cp);
      atomicAdd(&sh.h.cnt[b], 1u);
      const uint64_t w = static_cast<uint64_t>(__fmul_rn(weight(v[e], top, c), kMassScale));
      const uint32_t wl = static_cast<uint32_t>(w);
      if (w) {
        const uint32_t old = atomicAdd(&sh.h.lo[b], wl);
        const uint32_t up = static_cast<uint32_t>(w >> 32) + (old + wl < old ? 1u : 0u);
        if (up) atomicAdd(&sh.h.hi[b], up);
      }
    }
  });
  __syncthreads();
  cluster_sync();
  // rank r sums bins r * per ... over all ranks into its own copy, for rank 0 to read
  const int per = kBins / size;
  for (int i = threadIdx.x; i < per; i += kSelThreads) {
    const int b = rank * per + i;
    uint32_t n = 0;
    uint64_t m = 0;
    for (uint32_t k = 0; k < size; ++k) {
      n += peer_ld32(peer(&sh.h.cnt[b], k));
      m += peer_ld32(peer(&sh.h.lo[b], k)) + (static_cast<uint64_t>(peer_ld32(peer(&sh.h.hi[b], k))) << 32);
    }
    // bin b of another rank's copy is read by this rank alone: overwrite rank 0's
    peer_st32(peer(&sh.h.cnt[b], 0), n);
    peer_st32(peer(&sh.h.lo[b], 0), static_cast<uint32_t>(m));
    peer_st32(peer(&sh.h.hi[b], 0), static_cast<uint32_t>(m >> 32));
  }
  cluster_sync();
  if (rank == 0) {
    // every thread: eight bins; prefix over the threads; the thread that holds the cut says so
    constexpr int PT = kBins / kSelThreads;
    const int b0 = threadIdx.x * PT;
    uint32_t n = 0;
    uint64_t m = 0;
    for (int k = 0; k < PT; ++k) {
      n += sh.h.cnt[b0 + k];
      m += sh.h.lo[b0 + k] + (static_cast<uint64_t>(sh.h.hi[b0 + k]) << 32);
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t sn = n;
    uint64_t sm = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t xn = __shfl_up_sync(0xffffffffu, sn, o);
      const uint64_t xm = __shfl_up_sync(0xffffffffu, sm, o);
      if (lane >= o) {
        sn += xn;
        sm += xm;
      }
    }
    if (lane == 31) {
      sh.redi[warp] = static_cast<int>(sn);
      sh.redu[warp] = sm;
    }
    __syncthreads();
    uint32_t an = sh.above_cnt + sn - n;
    uint64_t am = sh.above_mass + sm - m, total = sh.above_mass;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < warp) {
        an += sh.redi[w];
        am += sh.redu[w];
      }
      total += sh.redu[w];
    }
    if (!first) total = sh.total_mass;  // the whole universe's, from the first pass
    const double want = static_cast<double>(share) * static_cast<double>(total);
    __syncthreads();
    if (threadIdx.x == 0) sh.total_mass = total;
    // the last non-empty bin before which the criterion still holds
    int cut = -1;
    uint32_t cut_n = 0, cut_in = 0;
    uint64_t cut_m = 0;
    for (int k = 0; k < PT; ++k) {
      const uint32_t bn = sh.h.cnt[b0 + k];
      if (bn) {
        const bool holds = by_count ? an < static_cast<uint32_t>(target)
                                    : an == 0 || static_cast<double>(am) < want;
        if (holds) {
          cut = b0 + k;
          cut_n = an;
          cut_m = am;
          cut_in = bn;
        }
      }
      an += bn;
      am += sh.h.lo[b0 + k] + (static_cast<uint64_t>(sh.h.hi[b0 + k]) << 32);
    }
    const int last = block_reduce(cut, sh.redi, [](int a, int b) { return max(a, b); });
    if (last < 0 && threadIdx.x == 0) sh.in_cnt = 0;  // an empty universe
    if (cut == last && cut >= 0) {
      sh.above_cnt = cut_n;
      sh.above_mass = cut_m;
      sh.in_cnt = cut_in;
      // its tokens: a range of comp
      if (first) {
        // smallest and largest key of the bin, by bisection (the bin number falls with the key)
        auto at = [&](uint32_t key) { return bin(value_of(key), 0); };
        uint32_t a = kKeyLowest, b = key_of(top);  // at(b) <= cut
        while (a < b) {                               // smallest key with at(key) <= cut
          const uint32_t mid = a + (b - a) / 2;
          if (at(mid) <= cut) b = mid;
          else a = mid + 1;
        }
        const uint32_t kmin = a;
        a = kmin;
        b = key_of(top);
        while (a < b) {  // largest key with at(key) >= cut
          const uint32_t mid = a + (b - a + 1) / 2;
          if (at(mid) >= cut) a = mid;
          else b = mid - 1;
        }
        sh.clo = max(static_cast<uint64_t>(kmin) << 32, ulo);
        sh.chi = (static_cast<uint64_t>(a) << 32) | 0xFFFFFFFFu;
      } else {
        const uint64_t hi = bin.chi - (static_cast<uint64_t>(cut) << bin.shift);
        const uint64_t span = (1ull << bin.shift) - 1;
        sh.chi = hi;
        sh.clo = max(max(bin.clo, hi > span ? hi - span : 0), ulo);
      }
    }
    __syncthreads();
  }
  cluster_sync();
  if (rank != 0 && threadIdx.x == 0) {
    sh.clo = peer_ld64(peer(&sh.clo, 0));
    sh.chi = peer_ld64(peer(&sh.chi, 0));
    sh.above_mass = peer_ld64(peer(&sh.above_mass, 0));
    sh.above_cnt = peer_ld32(peer(&sh.above_cnt, 0));
    sh.in_cnt = peer_ld32(peer(&sh.in_cnt, 0));
  }
  __syncthreads();
  cluster_sync();  // rank 0 goes on to change them
}

// The tokens of [clo, chi] into rank 0's list and, with SCORE, the race over
// the tokens above chi that min-p keeps, with their mass.
template <bool VEC, bool SCORE>
__device__ void collect(SelShared& sh, const float* row, int V, const RowParam& p, Race& race, uint64_t& mass) {
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const float c = __fdiv_rn(kLog2e, p.temp), inv_t = __fdiv_rn(1.f, p.temp), top = sh.top;
  const uint64_t clo = sh.clo, chi = sh.chi;
  if (rank == 0 && threadIdx.x == 0) sh.n = 0;
  cluster_sync();
  const uint32_t n_at = peer(&sh.n, 0), list_at = peer(sh.l.comp, 0);
  mass = 0;
  for_slice<VEC>(row, V, rank, size, [&](const float4& x, int q) {
    const float v[4] = {x.x, x.y, x.z, x.w};
    bool up[4], any = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint64_t cp = comp_of(v[e], q * 4 + e);
      up[e] = false;
      if (cp < clo) continue;
      if (cp <= chi) {
        const uint32_t at = peer_add32(n_at, 1u);
        if (at < kList) peer_st64(list_at + 8 * at, cp);
      } else if (SCORE && min_p_keeps(v[e], top, p.temp, p.log_min_p)) {
        up[e] = any = true;
        mass += static_cast<uint64_t>(__fmul_rn(weight(v[e], top, c), kMassScale));
      }
    }
    if (SCORE && any) {
      const uint4 w = philox_block(p.seed, p.step, static_cast<uint32_t>(q));
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (up[e]) race.token(v[e], q * 4 + e, word_of(w, e), p.temp, inv_t);
    }
  });
  cluster_sync();
}

// A row whose cut lies below the lists: the whole cluster re-reads it.
template <bool VEC>
__device__ void wide_row(SelShared& sh, const SelectArgs& a, const RowParam& p, int r) {
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const float* row = a.logits + r * a.ld;
  const int V = a.V;
  uint64_t ulo = static_cast<uint64_t>(kKeyLowest) << 32;  // the universe: comp >= ulo
  Race race;
  uint64_t mass = 0;
  auto restart = [&] {
    if (threadIdx.x == 0) {
      sh.clo = ulo;
      sh.chi = ~0ull;
      sh.above_mass = 0;
      sh.above_cnt = 0;
      sh.in_cnt = 0;
    }
    __syncthreads();
  };
  auto narrow = [&](bool by_count, float share) {
    restart();
    bool first = true;
    do {
      histogram_cut<VEC>(sh, row, V, p, first, ulo, by_count, p.top_k, share);
      first = false;
    } while (sh.in_cnt > kList);
  };
  const bool has_p = p.top_p < 1.f;
  double z = 0;  // mass that top-p is a share of, where top-k cut first
  if (p.top_k > 0) {
    narrow(true, 0.f);
    if (has_p) {  // top-k exactly, then top-p within it
      collect<VEC, false>(sh, row, V, p, race, mass);
      if (rank == 0) {
        sort_desc(sh.l.comp, sh.n);
        if (threadIdx.x == 0) {
          const int last = min(sh.n, static_cast<int>(p.top_k - sh.above_cnt)) - 1;
          sh.last_comp = sh.l.comp[max(last, 0)];
        }
        __syncthreads();
      }
      cluster_sync();
      ulo = peer_ld64(peer(&sh.last_comp, 0));
      cluster_sync();
    }
  }
  if (has_p) {
    narrow(false, p.top_p);
    z = static_cast<double>(sh.total_mass);  // rank 0's
  } else if (p.top_k == 0) {  // min-p alone: every token is "above", nothing undecided
    if (threadIdx.x == 0) {
      sh.clo = ulo;
      sh.chi = ulo - 1;
      sh.above_cnt = 0;
      sh.above_mass = 0;
    }
    __syncthreads();
  }
  const uint64_t above = sh.above_mass;  // of the tokens above the undecided bin
  const uint32_t above_n = sh.above_cnt;
  collect<VEC, true>(sh, row, V, p, race, mass);
  mass = block_reduce(mass, sh.redu, [](uint64_t x, uint64_t y) { return x + y; });
  race.warp_reduce();
  if ((threadIdx.x & 31) == 0) {
    sh.redf[threadIdx.x >> 5] = race.best;
    sh.redi[threadIdx.x >> 5] = race.best_i;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kSelThreads / 32; ++w) race.take(sh.redf[w], sh.redi[w]);
    peer_st32(peer(&sh.r_best[rank], 0), __float_as_uint(race.best));
    peer_st32(peer(&sh.r_best_i[rank], 0), static_cast<uint32_t>(race.best_i));
    peer_st64(peer(&sh.r_mass[rank], 0), mass);
  }
  cluster_sync();  // the last access to another CTA's memory
  if (rank != 0) return;
  Race best;
  uint64_t kept_mass = 0;
  for (uint32_t k = 0; k < size; ++k) {
    if (better(sh.r_best[k], sh.r_best_i[k], best.best, best.best_i)) {
      best.best = sh.r_best[k];
      best.best_i = sh.r_best_i[k];
    }
    kept_mass += sh.r_mass[k];
  }
  const int n = sh.n;
  const double unit = 1.0 / kMassScale, base = static_cast<double>(above) * unit;
  const double want = static_cast<double>(p.top_p) * (z * unit);
  sort_desc(sh.l.comp, n);
  prefix_mass(sh, n, sh.top, p.temp, base);
  int kept = 0;
  for (int j = threadIdx.x; j < n; j += kSelThreads) {
    const float l = value_of(static_cast<uint32_t>(sh.l.comp[j] >> 32));
    const bool in_k = has_p || p.top_k == 0 || above_n + j < static_cast<uint32_t>(p.top_k);
    const bool in_p = !has_p || above_n + j == 0 || (j == 0 ? base : sh.l.pre[j - 1]) < want;
    kept += in_k && in_p && min_p_keeps(l, sh.top, p.temp, p.log_min_p);
  }
  kept = block_reduce(kept, sh.redi, [](int x, int y) { return x + y; });
  const double total = static_cast<double>(kept_mass) * unit + (kept > 0 ? sh.l.pre[kept - 1] - base : 0.0);
  choose(sh, p, kept, best, total, sh.top, row, a.tokens + r, a.logprobs ? a.logprobs + r : nullptr);
}

template <int N, bool VEC>
__global__ void __launch_bounds__(kSelThreads)
    filter_select_kernel(const __grid_constant__ RowParams<N> params, SelectArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SelShared& sh = *reinterpret_cast<SelShared*>(smem_raw);
  float* seg_max = reinterpret_cast<float*>(smem_raw + sizeof(SelShared));  // [nseg]
  int* seg_n = reinterpret_cast<int*>(seg_max + a.nseg);                     // [nseg]
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const int r = blockIdx.x / size;
  const RowParam p = params.r[r];
  const int mode = row_mode(p);
  pdl_wait();
  pdl_trigger();
  if (mode != ROW_FILTER && rank != 0) return;
  const float* row = a.logits + r * a.ld;
  bool wide = false;
  if (rank == 0) {
    const SegOut* segs = a.segs + static_cast<size_t>(r) * a.nseg;
    float top = -INFINITY;
    uint32_t thr = kKeyLowest;
    Race race;
    for (int i = threadIdx.x; i < a.nseg; i += kSelThreads) {
      const SegOut s = segs[i];
      seg_max[i] = s.max;
      seg_n[i] = s.count;
      top = fmaxf(top, s.max);
      thr = max(thr, s.thr);
      if (better(s.best, s.best_i, race.best, race.best_i)) {
        race.best = s.best;
        race.best_i = s.best_i;
      }
    }
    top = block_reduce(top, sh.redf, [](float x, float y) { return fmaxf(x, y); });
    double z = 0;
    if (mode != ROW_GREEDY) {
      const float c = __fdiv_rn(kLog2e, p.temp);
      for (int i = threadIdx.x; i < a.nseg; i += kSelThreads)
        z += static_cast<double>(segs[i].sum) * static_cast<double>(weight(seg_max[i], top, c));
      z = block_reduce(z, sh.redd, [](double x, double y) { return x + y; });
    }
    if (mode != ROW_FILTER || top == -INFINITY) {
      choose(sh, p, 0, race, mode == ROW_GREEDY ? 1.0 : z, top, row, a.tokens + r, nullptr);
      if (threadIdx.x == 0 && a.logprobs) {
        const int tok = a.tokens[r];
        const float l = row[tok], d = l == top ? 0.f : __fdiv_rn(__fsub_rn(l, top), p.temp);
        a.logprobs[r] = mode != ROW_FREE || top == -INFINITY ? 0.f : __fsub_rn(d, log1pf(static_cast<float>(z - 1.0)));
      }
      if (mode != ROW_FILTER) return;
    }
    thr = block_reduce(thr, reinterpret_cast<uint32_t*>(sh.redi), [](uint32_t x, uint32_t y) { return max(x, y); });
    const uint32_t floor = thr;  // every logit from here on is listed
    const bool all = floor <= kKeyLowest;  // the lists hold every finite logit
    // First as many candidates as there are large segment maxima (at least the
    // first `want` tokens are among those at or above the want-th largest), then,
    // if that does not decide the row, every listed one.
    wide = top > -INFINITY;  // without any finite logit the choice has been made
    for (int level = 0; level < 2 && wide; ++level) {
      uint32_t from = floor;
      if (level == 0) {
        const int want = min(p.top_k > 0 ? min(p.top_k, 64) : 48, a.nseg);
        uint32_t mine = 0;  // the want-th largest segment maximum's key
        for (int i = threadIdx.x; i < a.nseg; i += kSelThreads) {
          int above = 0;
          const float m = seg_max[i];
          for (int j = 0; j < a.nseg; ++j) above += seg_max[j] > m || (seg_max[j] == m && j < i);
          if (above == want - 1) mine = key_of(m);
        }
        from = max(block_reduce(mine, reinterpret_cast<uint32_t*>(sh.redi),
                                [](uint32_t x, uint32_t y) { return max(x, y); }),
                   floor);
        if (from == floor) continue;
      }
      if (threadIdx.x == 0) sh.n = 0;
      __syncthreads();
      const int lane = threadIdx.x & 31;
      for (int i = threadIdx.x >> 5; i < a.nseg; i += kSelThreads / 32) {
        if (key_of(seg_max[i]) < from) continue;
        const uint64_t* list = a.lists + (static_cast<size_t>(r) * a.nseg + i) * kSegCap;
        for (int k = lane; k < seg_n[i]; k += 32) {
          const uint64_t cp = list[k];
          if (static_cast<uint32_t>(cp >> 32) >= from) {
            const int at = atomicAdd(&sh.n, 1);
            if (at < kList) sh.l.comp[at] = cp;
          }
        }
      }
      __syncthreads();
      const int n = sh.n;
      if (n > kList || n == 0) continue;  // too many candidates, or none listed (ties)
      const bool complete = all && from == floor;
      sort_desc(sh.l.comp, n);
      prefix_mass(sh, n, top, p.temp, 0.0);
      const int lim = p.top_k > 0 ? min(p.top_k, n) : n;
      const bool k_known = complete || p.top_k <= n;  // with top_k on: the list holds all of its tokens
      const bool has_p = p.top_p < 1.f;
      if (p.top_k > 0 && has_p && !k_known) continue;
      const double share = static_cast<double>(p.top_p) * (p.top_k > 0 ? sh.l.pre[lim - 1] : z);
      int kept = 0;
      for (int j = threadIdx.x; j < lim; j += kSelThreads) {
        const float l = value_of(static_cast<uint32_t>(sh.l.comp[j] >> 32));
        kept += (!has_p || j == 0 || sh.l.pre[j - 1] < share) && min_p_keeps(l, top, p.temp, p.log_min_p);
      }
      kept = block_reduce(kept, sh.redi, [](int x, int y) { return x + y; });
      const bool decided = complete || kept < n || (p.top_k > 0 && p.top_k <= n) ||
                           (has_p && sh.l.pre[lim - 1] >= share);
      if (!decided) continue;
      wide = false;
      choose(sh, p, kept, Race(), kept > 0 ? sh.l.pre[kept - 1] : 1.0, top, row, a.tokens + r,
             a.logprobs ? a.logprobs + r : nullptr);
    }
    if (threadIdx.x == 0) {
      sh.go = wide;
      sh.top = top;
    }
  }
  cluster_sync();
  if (rank != 0) {
    wide = peer_ld32(peer(&sh.go, 0)) != 0;
    const float top = __uint_as_float(peer_ld32(peer(&sh.top, 0)));
    __syncthreads();
    if (threadIdx.x == 0) sh.top = top;
  }
  cluster_sync();
  if (wide) wide_row<VEC>(sh, a, p, r);
}

template <int N>
int launch_filter_n(const SampleFilterArgs& a, int r0, int rows, cudaStream_t s) {
  RowParams<N> params;
  for (int i = 0; i < rows; ++i) {
    const vd_sampler& sp = a.samplers[r0 + i];
    RowParam& p = params.r[i];
    p.seed = sp.seed;
    p.step = sp.step;
    p.temp = sp.temperature;
    p.top_p = 1.f;
    p.log_min_p = -INFINITY;
    p.top_k = 0;
    if (a.filters) {
      const vd_filter& f = a.filters[r0 + i];
      p.top_k = f.top_k > 0 && f.top_k < a.V ? f.top_k : 0;
      p.top_p = f.top_p;
      p.log_min_p = f.min_p > 0.f ? static_cast<float>(log(static_cast<double>(f.min_p))) : -INFINITY;
    }
  }
  for (int i = rows; i < N; ++i) params.r[i] = RowParam{};
  const int nseg = (a.V + kSeg - 1) / kSeg;
  // a list's length in all: about 1500 candidates a row reach the largest threshold
  const int keep = nseg <= 128 ? 16 : nseg <= 256 ? 8 : nseg <= 512 ? 4 : 2;
  SegOut* segs = static_cast<SegOut*>(a.workspace) + static_cast<size_t>(r0) * nseg;
  uint64_t* lists = reinterpret_cast<uint64_t*>(static_cast<SegOut*>(a.workspace) + static_cast<size_t>(a.R) * nseg) +
                    static_cast<size_t>(r0) * nseg * kSegCap;
  const float* logits = a.logits + r0 * a.ld;
  const bool vec = (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0 && a.ld % 4 == 0;
  VD_CUDA_TRY(launch_k(vec ? filter_scan_kernel<N, true> : filter_scan_kernel<N, false>,
                       dim3((nseg + kScanThreads / 32 - 1) / (kScanThreads / 32), rows), dim3(kScanThreads), 0, s, params,
                       logits, a.V, a.ld, nseg, keep, segs, lists));
  SelectArgs sel{};
  sel.logits = logits;
  sel.ld = a.ld;
  sel.V = a.V;
  sel.nseg = nseg;
  sel.segs = segs;
  sel.lists = lists;
  sel.tokens = a.tokens + r0;
  sel.logprobs = a.logprobs ? a.logprobs + r0 : nullptr;
  const int cluster = rows <= 64 ? 8 : 4;
  const size_t smem = sizeof(SelShared) + static_cast<size_t>(nseg) * 8;
  auto k = vec ? filter_select_kernel<N, true> : filter_select_kernel<N, false>;
  if (smem > 48 * 1024)
    VD_CUDA_TRY(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(rows * cluster);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  VD_CUDA_TRY(cudaLaunchKernelEx(&cfg, k, params, sel));
  return VD_OK;
}

}  // namespace

size_t sample_filter_workspace(int R, int V) {
  const size_t nseg = (static_cast<size_t>(V) + kSeg - 1) / kSeg;
  return static_cast<size_t>(R) * nseg * (sizeof(SegOut) + kSegCap * sizeof(uint64_t));
}

int launch_sample_filter(const SampleFilterArgs& a, cudaStream_t s) {
  // the rows' parameters travel in the kernel parameters (40 bytes each)
  for (int r0 = 0; r0 < a.R; r0 += 512) {
    const int rows = std::min(512, a.R - r0);
    const int rc = rows <= 16 ? launch_filter_n<16>(a, r0, rows, s)
                   : rows <= 128 ? launch_filter_n<128>(a, r0, rows, s)
                                 : launch_filter_n<512>(a, r0, rows, s);
    if (rc) return rc;
  }
  return VD_OK;
}

}  // namespace vd
