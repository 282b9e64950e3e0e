// Token choice with temperature, top-k, top-p and min-p.
//
// A row's kept tokens are a prefix of its tokens in descending order (ties:
// lower index first), cut by the filters that are on: the top_k first; those
// before which the probability mass is below top_p; those whose probability is
// at least min_p of the largest.  The choice is the Gumbel-max choice of
// sampler.cu over the kept tokens, with the same random numbers and the same
// scores, so that a row without filters gets exactly vd_sample's token.
//
// Almost every row is decided by a few dozen of its V logits.
//
//   scan     reads the logits once, at memory speed.  A warp takes a segment
//            of 1024, finds its maximum, its sum of exponentials and a
//            threshold that a few of its logits reach (the smallest maximum of
//            a few groups of lanes), and writes the logits from that threshold
//            on to a short list: every logit at or above the largest threshold
//            of a row's segments is then in a list.
//   select   one CTA per row takes as many listed candidates as it needs and
//            finds the cut among them: up to 128 sorted, more by bins of value
//            (only the cut's bin needs an order).
//
// A row whose cut lies below the lists (flat distributions, logits sorted
// along the vocabulary) is "wide".  Two more kernels, whose CTAs take (wide
// row, part of it) items, read it again:
//
//   count    a histogram of 4096 bins of value, tokens and their mean place in
//            the bin; the last CTA of a row estimates each bin's mass from
//            them and picks the window of bins that holds the cut;
//   collect  scores every token above the window and sums their mass, and
//            lists the tokens inside it; the last CTA of a row sorts those,
//            checks that the cut is among them and chooses.
//
// What that cannot settle (a window of more than kList tokens, top-p within a
// top_k beyond the lists) one CTA settles by exact histograms over the
// (value, index) order, refined until the cut's bin fits the list.
//
// Masses are integers, one per token whichever kernel adds it: nothing depends
// on timing, on the CTAs that share a row or on the other rows of the call.
//
// Measured: one row of 128256, top-k 50 and top-p 0.9, 13 us (host 11); 256
// rows of mixed settings 83 to 101 us by seed, 61 rows of 262144 with nuclei of
// tens of thousands of tokens 134 to 146 us.  The floor is one read of the logits, 19.4 us and
// 9.5 us; each kernel's comment says what it spends.
#include <float.h>
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
constexpr int kScanCtas = 4;      // resident per SM
constexpr int kSelThreads = 256;
constexpr int kBins = 2048;       // exact histogram: counts and masses, by (value, index) order
constexpr int kCountBins = 4096;  // a wide row's histogram, by value
constexpr float kBinNats = 24.f;  // its range below the largest logit at most, in units of T
constexpr int kList = 2048;       // candidates that a CTA sorts
constexpr int kListBins = 1024;   // an unsorted list's bins of value
constexpr int kCutList = 512;     // candidates of the cut's bin
constexpr int kChunk = 4096;      // a wide row's work item has this many tokens or more
constexpr int kCountTurn = 8192;  // tokens that the packed counters of `count` hold
constexpr int kScanRows = 512;    // rows of a scan launch (their parameters travel with it: 34 bytes each)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMassScale = 68719476736.f;  // 2^36

enum RowMode { ROW_GREEDY = 0, ROW_FREE = 1, ROW_FILTER = 2 };

struct RowParam {
  uint64_t seed, step;
  float temp, top_p, log_min_p;  // top_p >= 1: off; log_min_p = -inf: off
  int top_k;                     // 0: off
};
template <int N>
struct RowParams {
  RowParam r[N];
  short row[N];  // the row of each, after the launch's first
};
__host__ __device__ __forceinline__ int row_mode(const RowParam& p) {
  if (!(p.temp > 0.f)) return ROW_GREEDY;
  return p.top_k > 0 || p.top_p < 1.f || p.log_min_p > -INFINITY ? ROW_FILTER : ROW_FREE;
}

// Whether a row's whole mass is asked for: top-p over every token, or the
// log-probability of an unfiltered choice.
__host__ __device__ __forceinline__ bool needs_mass(const RowParam& p) {
  return p.temp > 0.f && p.top_k == 0 && (p.top_p < 1.f || !(p.log_min_p > -INFINITY));
}

// What the scan leaves of a segment.
struct __align__(16) SegOut {
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
// infinite), 0 for NaN.  Every token's mass is made of this (collect_quads has
// it inline) and of mass_rate(T), c kept finite: a difference of zero times an
// infinite c, as of T below float32's normal range, is no zero.
__device__ __forceinline__ float mass_rate(float t) { return fminf(__fdiv_rn(kLog2e, t), FLT_MAX); }
__device__ __forceinline__ float weight(float l, float m, float c) {
  const float w = ex2(__fmul_rn(__fsub_rn(l, m), c));
  return l == m ? 1.f : w == w ? w : 0.f;
}

// One copy of the score's two logarithms and division per kernel: the streams
// below call it for few tokens, from many unrolled places.
__device__ __noinline__ float score_of(float l, uint32_t word, float t) { return gumbel_score(l, word, t); }

// Masses are 64-bit integers in units of 2^-36 of the largest token's: sums
// are exact in any order (V <= 2^21 tokens of mass at most 1: below 2^57), and
// the GPU's few double-precision units stay out of it.
__device__ __forceinline__ uint64_t fixed(float w) { return static_cast<uint64_t>(__fmul_rn(w, kMassScale)); }
// Sums of fixed(w), w in [0, 1], without its conversions: adding 32 rounded down
// leaves floor(2^18 w) in the low bits of the float, adding 2^-13 to what is
// left over (exact) leaves the next 18 bits.  The sums of the bits are taken
// modulo 2^32 and the constants' bits off again: exact for 2^13 tokens.  So a
// token's mass is the same whichever kernel, part and thread adds it.
struct MassSum {
  uint32_t hi = 0, lo = 0;
  __device__ __forceinline__ void add4(const float (&w)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float t = __fadd_rd(w[e], 32.f), r = __fsub_rn(w[e], __fsub_rn(t, 32.f));
      hi += __float_as_uint(t);
      lo += __float_as_uint(__fadd_rd(r, 1.220703125e-4f));
    }
    hi -= 4u * 0x42000000u;
    lo -= 4u * 0x39000000u;
  }
  __device__ __forceinline__ uint64_t value() const { return (static_cast<uint64_t>(hi) << 18) + lo; }
};
__device__ __forceinline__ uint64_t share_of(float top_p, uint64_t mass) {
  return static_cast<uint64_t>(static_cast<double>(top_p) * static_cast<double>(mass));
}

// The best Gumbel score of a stream of tokens, without the two logarithms
// for tokens that cannot win: G = -log(-log u) <= -log(1 - u), so a token
// beats `best` only if 1 - u <= exp(x - best).  The test errs on the side of
// scoring: its margin (1e-3 and 2^-20 of the magnitudes) covers the rounding
// of the test, of l / T and of the score, so the winner is the one that
// scoring every token finds.  It costs six instructions a token; 1 - u is
// read off the random word as the float 1 + 2^-23 (~word >> 9).
struct Race {
  float best = -INFINITY;
  int best_i = INT_MAX;
  float k0 = INFINITY;  // -log2(e) (best - margin)
  __device__ __forceinline__ void set_bound() {
    const float margin = __fmaf_rn(fabsf(best), 9.5367431640625e-7f, 1.1e-3f);
    k0 = __fmul_rn(__fsub_rn(margin, best), kLog2e);
  }
  __device__ __forceinline__ void take(float v, int i) {
    if (better(v, i, best, best_i)) {
      best = v;
      best_i = i;
      set_bound();
    }
  }
  // The same with the exponential at hand: w = exp((l - top) / T), ratio from
  // `ratio_to(top, c)` for the current bound.
  __device__ __forceinline__ float ratio_to(float top, float c) const { return ex2(__fmaf_rn(top, c, k0)); }
  __device__ __forceinline__ bool may_win(float w, float ratio, uint32_t word) const {
    const float rest = __uint_as_float((~word >> 9) | 0x3F800000u);
    return !(rest > __fadd_rn(__fmul_rn(w, ratio), 1.0000002384185791015625f));
  }
  // c = log2(e) / T
  __device__ __forceinline__ void token(float l, int i, uint32_t word, float t, float c) {
    const float a = ex2(__fmaf_rn(l, c, k0));
    const float rest = __uint_as_float((~word >> 9) | 0x3F800000u);
    if (!(rest > __fadd_rn(a, 1.0000002384185791015625f))) take(score_of(l, word, t), i);
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
    set_bound();
  }
};

// philox_block with each 32 x 32 product as one wide multiply and the key
// schedule shared by a thread's blocks (the same words).
struct Philox {
  uint32_t k0, k1, c1, c2;
  __device__ __forceinline__ explicit Philox(const RowParam& p)
      : k0(static_cast<uint32_t>(p.seed)), k1(static_cast<uint32_t>(p.seed >> 32)), c1(static_cast<uint32_t>(p.step)),
        c2(static_cast<uint32_t>(p.step >> 32)) {}
  __device__ __forceinline__ uint4 block(uint32_t blk) const {
    uint32_t x = blk, y = c1, z = c2, w = 0x5644u;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * x, b = static_cast<uint64_t>(0xCD9E8D57u) * z;
      x = static_cast<uint32_t>(b >> 32) ^ y ^ (k0 + r * 0x9E3779B9u);
      y = static_cast<uint32_t>(b);
      z = static_cast<uint32_t>(a >> 32) ^ w ^ (k1 + r * 0xBB67AE85u);
      w = static_cast<uint32_t>(a);
    }
    return make_uint4(x, y, z, w);
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

// What one row's wide kernels share.
struct __align__(16) WideState {
  uint64_t z;            // the row's whole mass
  uint64_t clo, chi;     // the window: a range of comp, inclusive
  float top;             // largest logit
  float least;           // smallest value that min-p keeps
  uint32_t above_n;      // tokens above the window
  uint32_t in_n;         // tokens inside it; more than kList: no usable window
  uint32_t arrived[2];   // CTAs done, per kernel
  int n;                 // tokens listed
  float bound;           // a score that some kept token has: only tokens that reach it matter
  float range;           // of the bins of `count`, down from `top`
};
struct __align__(16) ChunkOut {
  uint64_t mass;           // of an item's tokens above the window (and at least `least`)
  float best;
  int best_i;
};

// The workspace of R rows.
struct Space {
  RowParam* params;      // [R]
  SegOut* segs;          // [R][nseg]
  uint64_t* lists;       // [R][nseg][kSegCap]
  WideState* wide;       // [R]
  ChunkOut* chunks;      // [R][nchunk]
  uint64_t* window;      // [R][kList]
  unsigned long long* count;  // [R][kCountBins] tokens << 32 | the sum of their places in the bin, in 32nds
  int* wide_rows;        // [R]
  int* n_wide;           // wide rows; then the next item of `count` and of `collect`
};
inline __host__ size_t space_of(Space* sp, void* base, int R, int nseg, int nchunk) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 127) / 128 * 128;
    return static_cast<char*>(base) + o;
  };
  const size_t r = R;
  sp->n_wide = reinterpret_cast<int*>(take(3 * sizeof(int)));
  sp->wide_rows = reinterpret_cast<int*>(take(r * sizeof(int)));
  sp->params = reinterpret_cast<RowParam*>(take(r * sizeof(RowParam)));
  sp->wide = reinterpret_cast<WideState*>(take(r * sizeof(WideState)));
  sp->segs = reinterpret_cast<SegOut*>(take(r * nseg * sizeof(SegOut)));
  sp->lists = reinterpret_cast<uint64_t*>(take(r * nseg * kSegCap * sizeof(uint64_t)));
  sp->chunks = reinterpret_cast<ChunkOut*>(take(r * nchunk * sizeof(ChunkOut)));
  sp->window = reinterpret_cast<uint64_t*>(take(r * kList * sizeof(uint64_t)));
  sp->count = reinterpret_cast<unsigned long long*>(take(r * kCountBins * sizeof(unsigned long long)));
  return off;
}

// ---------------------------------------------------------------- scan
// A warp walks over (row, segment) items.  Bound by instruction issue next to
// memory: 131 MB in 36 us (3.6 TB/s), 640 warp instructions per segment, issue 56
// % active; copies through shared memory one item ahead measured 35 us, L2
// prefetches of the next item nothing.  first: the call's first scan launch.
// The others depend on no earlier kernel but through it, so they wait for
// their predecessor at their end: they run next to it, and whatever waits for
// the last one waits for all.
template <int N, bool VEC>
__global__ void __launch_bounds__(kScanThreads, kScanCtas)
    filter_scan_kernel(const __grid_constant__ RowParams<N> params, const float* __restrict__ logits, int V,
                       long long ld, int nseg, int groups, bool first, Space sp, int r0, int rows) {
  if (first) pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0) {
    for (int r = threadIdx.x; r < rows; r += kScanThreads) sp.params[r0 + params.row[r]] = params.r[r];
    if (first && threadIdx.x < 3) sp.n_wide[threadIdx.x] = 0;
  }
  const int items = rows * nseg;
  for (int item = blockIdx.x * (kScanThreads / 32) + warp; item < items; item += gridDim.x * (kScanThreads / 32)) {
    const int r = item / nseg, seg = item % nseg, row_i = r0 + params.row[r], i0 = seg * kSeg + lane * 4;
    const float* row = logits + row_i * ld;
    float v[8][4];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float4 x = load4<VEC>(row, i0 + q * 128, V);
      v[q][0] = x.x;
      v[q][1] = x.y;
      v[q][2] = x.z;
      v[q][3] = x.w;
    }
    const RowParam& p = params.r[r];
    const int mode = row_mode(p);
    float lm = -INFINITY;
#pragma unroll
    for (int q = 0; q < 8; ++q) lm = fmaxf(lm, fmaxf(fmaxf(v[q][0], v[q][1]), fmaxf(v[q][2], v[q][3])));
    float m = lm;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    SegOut out{};
    out.max = m;
    out.thr = kKeyLowest;
    Race race;
    const float c = __fdiv_rn(kLog2e, p.temp);
    if (mode == ROW_GREEDY || m == -INFINITY) {
      // the lowest index among the maxima; a row of NaN and -inf has its lowest -inf
#pragma unroll
      for (int q = 7; q >= 0; --q)
#pragma unroll
        for (int e = 3; e >= 0; --e)
          if (v[q][e] == m) race.best_i = i0 + q * 128 + e;
      race.best = race.best_i == INT_MAX ? -INFINITY : m;
      race.warp_reduce();
    } else if (mode == ROW_FREE) {
      // each lane's largest logit first: the best of those 32 leaves few others to score
      const Philox ph(p);
      int at = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) at = v[q][e] == lm ? q * 128 + e : at;
      if (lm > -INFINITY) race.take(score_of(lm, word_of(ph.block(static_cast<uint32_t>(i0 + at) / 4), at & 3), p.temp), i0 + at);
      race.warp_reduce();
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int i = i0 + q * 128;
        const uint4 w = ph.block(static_cast<uint32_t>(i) / 4);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e < V) race.token(v[q][e], i + e, word_of(w, e), p.temp, c);
      }
      race.warp_reduce();
    } else {
      // The smallest of the maxima of `groups` groups of lanes: at least
      // `groups` logits reach it (about groups (ln(groups) + 0.58) of logits
      // in no order).  Where the list would be too long (one segment in 500),
      // half the groups, down to the maximum alone; if even that repeats too
      // often, nothing is listed.
      out.thr = key_of(m) + 1;
      uint64_t* list = sp.lists + (static_cast<size_t>(row_i) * nseg + seg) * kSegCap;
#pragma unroll 1
      for (int g = groups; g > 0; g >>= 1) {
        float low = lm;
        for (int o = 1; o < 32 / g; o <<= 1) low = fmaxf(low, __shfl_xor_sync(0xffffffffu, low, o));
        for (int o = 32 / g; o < 32; o <<= 1) low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
        const uint32_t t = max(key_of(low), kKeyLowest);  // -inf is never listed
        const float tv = value_of(t);
        uint32_t mine = 0;  // bit 4 q + e: v[q][e] is listed
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) mine |= v[q][e] >= tv ? 1u << (4 * q + e) : 0u;
        const int n = __popc(mine);
        int before = n;  // inclusive prefix sum over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += x;
        }
        const int total = __shfl_sync(0xffffffffu, before, 31);
        if (total > kSegCap) continue;
        before -= n;
        while (mine) {  // the few that are listed, read again from the cache (their registers have no run-time index)
          const int k = __ffs(mine) - 1, i = i0 + (k >> 2) * 128 + (k & 3);
          mine &= mine - 1;
          list[before++] = comp_of(row[i], i);
        }
        out.thr = t;
        out.count = total;
        break;
      }
    }
    if (needs_mass(p)) {
      const float rate = fminf(c, FLT_MAX);  // mass_rate
      float sum = 0.f;
      if (fabsf(m) < INFINITY) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sum = __fadd_rn(sum, fmaxf(ex2(__fmul_rn(__fsub_rn(v[q][e], m), rate)), 0.f));  // (the maximum drops NaN)
      } else {  // infinite logits share the mass
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum = __fadd_rn(sum, v[q][e] == m ? 1.f : 0.f);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
      out.sum = sum;
    }
    out.best = race.best;
    out.best_i = race.best_i;
    if (lane == 0) sp.segs[static_cast<size_t>(row_i) * nseg + seg] = out;
  }
  if (!first) pdl_wait();
}

// ---------------------------------------------------------------- shared by the deciding kernels
struct SelShared {
  union {
    struct {
      uint32_t cnt[kBins], lo[kBins], hi[kBins];  // tokens; masses as 64-bit integers in two words
    } h;
    uint32_t count[kCountBins];
    struct {
      uint64_t comp[kList];
      union {
        uint64_t pre[kList];  // masses up to and including each
        struct {              // or, for an unsorted list: bins of value, and the cut's bin
          uint32_t cnt[kListBins], lo[kListBins], hi[kListBins];
          uint64_t cut[kCutList];
        } b;
      };
    } l;
  };
  uint64_t redu[kSelThreads / 32];
  float redf[kSelThreads / 32];
  int redi[kSelThreads / 32];
  int n;                     // list entries
  int listed;                // and those of one item of a wide row
  int flag;
  uint64_t clo, chi;         // tokens of the undecided bin (comp range, inclusive)
  uint64_t above_mass;       // of the tokens above it
  uint64_t total_mass;
  uint32_t above_n, in_n;
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
__device__ __forceinline__ int block_sum(SelShared& sh, int v) {
  return block_reduce(v, sh.redi, [](int a, int b) { return a + b; });
}
__device__ __forceinline__ int block_max(SelShared& sh, int v) {
  return block_reduce(v, sh.redi, [](int a, int b) { return max(a, b); });
}
__device__ __forceinline__ uint64_t block_sum(SelShared& sh, uint64_t v) {
  return block_reduce(v, sh.redu, [](uint64_t a, uint64_t b) { return a + b; });
}
// The best of the block, on every thread.
__device__ __forceinline__ void block_best(SelShared& sh, Race& race) {
  race.warp_reduce();
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    sh.redf[threadIdx.x >> 5] = race.best;
    sh.redi[threadIdx.x >> 5] = race.best_i;
  }
  __syncthreads();
  for (int w = 0; w < kSelThreads / 32; ++w)
    if (better(sh.redf[w], sh.redi[w], race.best, race.best_i)) {
      race.best = sh.redf[w];
      race.best_i = sh.redi[w];
    }
}

// Bitonic sort, descending, of N = E * kSelThreads values, E consecutive ones
// per thread: distances below E inside the thread, below 32 E by shuffles,
// the rest through shared memory.
template <int E>
__device__ __forceinline__ void bitonic_desc(uint64_t (&v)[E], uint64_t* buf) {
  constexpr int N = E * kSelThreads;
  const int i0 = threadIdx.x * E;
#pragma unroll
  for (int k = 2; k <= N; k <<= 1) {
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      if (j >= 32 * E) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) buf[i0 + e] = v[e];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int i = i0 + e;
          const uint64_t o = buf[i ^ j];
          const bool larger = ((i & k) == 0) == ((i & j) == 0);
          v[e] = (o > v[e]) == larger ? o : v[e];
        }
      } else if (j >= E) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int i = i0 + e;
          const uint64_t o = __shfl_xor_sync(0xffffffffu, v[e], j / E);
          const bool larger = ((i & k) == 0) == ((i & j) == 0);
          v[e] = (o > v[e]) == larger ? o : v[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if ((e & j) == 0) {
            const bool down = ((i0 + e) & k) == 0;
            const uint64_t x = v[e], y = v[e ^ j];
            const bool swap = (y > x) == down;
            v[e] = swap ? y : x;
            v[e ^ j] = swap ? x : y;
          }
      }
    }
  }
}
template <int E>
__device__ void sort_n(uint64_t* comp, int n) {
  uint64_t v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = threadIdx.x * E + e < n ? comp[threadIdx.x * E + e] : 0;
  bitonic_desc<E>(v, comp);
  __syncthreads();
#pragma unroll
  for (int e = 0; e < E; ++e) comp[threadIdx.x * E + e] = v[e];
  __syncthreads();
}
// Sorts comp[0, n) in descending order (n <= kList, the values all different
// and above 0); the entries up to the next size are zeroed.
constexpr int kFew = kSelThreads / 2;
__device__ void sort_few(uint64_t* comp, int n) {
  if (n <= 32) {  // one warp, by shuffles
    if (threadIdx.x < 32) {
      uint64_t x = static_cast<int>(threadIdx.x) < n ? comp[threadIdx.x] : 0;
#pragma unroll
      for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
          const uint64_t o = __shfl_xor_sync(0xffffffffu, x, j);
          const bool larger = ((threadIdx.x & k) == 0) == ((threadIdx.x & j) == 0);
          x = (o > x) == larger ? o : x;
        }
      comp[threadIdx.x] = x;
    }
    __syncthreads();
  } else {  // by rank: each thread counts the values above its own
    const int i = threadIdx.x;
    const uint64_t mine = i < n ? comp[i] : 0;
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) rank += comp[j] > mine;
    __syncthreads();
    if (i < n) comp[rank] = mine;
    __syncthreads();
  }
}
__device__ void sort_desc(uint64_t* comp, int n) {
  static_assert(kList == 8 * kSelThreads, "sizes below");
  if (n <= kFew) {
    sort_few(comp, n);
  } else if (n <= kSelThreads) {
    sort_n<1>(comp, n);
  } else if (n <= 2 * kSelThreads) {
    sort_n<2>(comp, n);
  } else if (n <= 4 * kSelThreads) {
    sort_n<4>(comp, n);
  } else {
    sort_n<8>(comp, n);
  }
}

// A listed token's mass, by the same operations as in the kernels that stream
// the row: which of a row's tokens are listed depends on the kernels that a
// call has, and may not show in the sums.
__device__ __forceinline__ uint64_t mass_at(uint64_t comp, float top, float c) {
  return fixed(weight(value_of(static_cast<uint32_t>(comp >> 32)), top, c));
}
// pre[j] = base + the masses of comp[0 .. j].
__device__ void prefix_mass(SelShared& sh, int n, float top, float t, uint64_t base) {
  const int per = (n + kSelThreads - 1) / kSelThreads, j0 = threadIdx.x * per, j1 = min(n, j0 + per);
  const float c = mass_rate(t);
  uint64_t sum = 0;
  for (int j = j0; j < j1; ++j) {
    sum += mass_at(sh.l.comp[j], top, c);
    sh.l.pre[j] = sum;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t s = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t x = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += x;
  }
  __syncthreads();
  if (lane == 31) sh.redu[warp] = s;
  __syncthreads();
  uint64_t off = base + s - sum;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w)
    if (w < warp) off += sh.redu[w];
  for (int j = j0; j < j1; ++j) sh.l.pre[j] += off;
  __syncthreads();
}

__device__ __forceinline__ bool min_p_keeps(float l, float top, float t, float log_min_p) {
  return l == top || __fdiv_rn(__fsub_rn(l, top), t) >= log_min_p;
}
// The smallest key in [lo, hi] for which `holds`, which is true from some key
// on and at hi; a whole warp searches, 32 keys a round.
template <typename F>
__device__ __forceinline__ uint32_t first_key(uint32_t lo, uint32_t hi, F holds) {
  const uint32_t lane = threadIdx.x & 31;
  while (lo < hi) {
    const uint32_t step = (hi - lo) / 32 + 1;
    const uint64_t k = static_cast<uint64_t>(lo) + static_cast<uint64_t>(lane) * step;
    const uint32_t yes = __ballot_sync(0xffffffffu, k >= hi || holds(static_cast<uint32_t>(k)));
    const uint32_t f = __ffs(yes) - 1;  // lane 31's key is at or past hi unless a lane before it holds
    if (yes == 0) {
      lo = lo + 31 * step + 1;
    } else {
      const uint64_t at = static_cast<uint64_t>(lo) + static_cast<uint64_t>(f) * step;
      if (f > 0) lo = lo + (f - 1) * step + 1;
      hi = at < hi ? static_cast<uint32_t>(at) : hi;
      if (f == 0) break;
    }
  }
  return hi;
}
// The smallest value that min-p keeps (a whole warp).
__device__ float min_p_least(const RowParam& p, float top) {
  if (!(p.log_min_p > -INFINITY)) return value_of(kKeyLowest);
  return value_of(first_key(kKeyLowest, key_of(top),
                            [&](uint32_t k) { return min_p_keeps(value_of(k), top, p.temp, p.log_min_p); }));
}

struct Out {
  const float* logits;
  long long ld;
  int V, nseg, nchunk;
  int* tokens;
  float* logprobs;  // or null
};

// The choice among the first `kept` of the sorted list and `race` (the best
// of tokens outside it); mass: that of every kept token, relative to `top`.
__device__ void choose(SelShared& sh, const Out& o, int r, const RowParam& p, int kept, Race race, uint64_t mass,
                       float top, bool point) {
  const Philox ph(p);
  for (int j = threadIdx.x; j < kept; j += kSelThreads) {
    const uint64_t cp = sh.l.comp[j];
    const int i = index_of(cp);
    const uint4 w = ph.block(static_cast<uint32_t>(i) / 4);
    const float v = score_of(value_of(static_cast<uint32_t>(cp >> 32)), word_of(w, i & 3), p.temp);
    if (better(v, i, race.best, race.best_i)) {
      race.best = v;
      race.best_i = i;
    }
  }
  block_best(sh, race);
  if (threadIdx.x == 0) {
    const int tok = race.best_i == INT_MAX ? 0 : race.best_i;
    o.tokens[r] = tok;
    if (o.logprobs) {
      const float l = o.logits[r * o.ld + tok];
      const float d = l == top ? 0.f : __fdiv_rn(__fsub_rn(l, top), p.temp);
      // the largest token's mass is 1: log1p of the rest
      const float rest = __fmul_rn(static_cast<float>(mass - static_cast<uint64_t>(kMassScale)), 1.f / kMassScale);
      o.logprobs[r] = point ? 0.f : __fsub_rn(d, log1pf(rest));
    }
  }
}

// Quads [q0, q1) of a row: f(four logits, their index / 4), every lane of a
// warp taking part in each call (NaN past the end); end() after every kQuads.
constexpr int kQuads = 2;
template <bool VEC, typename F, typename E>
__device__ __forceinline__ void for_quads(const float* row, int V, int q0, int q1, F f, E end) {
  float4 x[kQuads];
  auto load = [&](int qb) {
#pragma unroll
    for (int u = 0; u < kQuads; ++u) {
      const int q = qb + u * kSelThreads + threadIdx.x;
      x[u] = q < q1 ? load4<VEC>(row, q * 4, V) : make_float4(NAN, NAN, NAN, NAN);
    }
  };
  load(q0);
  for (int qb = q0; qb < q1; qb += kQuads * kSelThreads) {
    float4 y[kQuads];
#pragma unroll
    for (int u = 0; u < kQuads; ++u) y[u] = x[u];
    load(qb + kQuads * kSelThreads);  // the next turn's, in flight during this one
#pragma unroll
    for (int u = 0; u < kQuads; ++u) f(y[u], qb + u * kSelThreads + static_cast<int>(threadIdx.x));
    end();
  }
}

// Tokens of quads [q0, q1): those of [clo, chi] go to `list` (its first kList
// places, counted in *n), and over those above chi of value at least `least`
// the mass is summed and, with SCORE, the race run.  mass: this thread's.
template <bool VEC, bool SCORE>
__device__ __forceinline__ void collect_quads(const float* row, int V, int q0, int q1, const RowParam& p, float top,
                                              float least, uint64_t clo, uint64_t chi, uint64_t* list, int* n,
                                              Race& race, uint64_t& mass) {
  const Philox ph(p);
  const float c = __fdiv_rn(kLog2e, p.temp), rate = fminf(c, FLT_MAX);  // mass_rate
  const float v_lo = value_of(static_cast<uint32_t>(clo >> 32)), v_hi = value_of(static_cast<uint32_t>(chi >> 32));
  float ratio = race.ratio_to(top, c);
  const float start = fmaxf(v_hi, least);  // no token below it counts
  MassSum part;                            // (V <= 2^21: at most 2^13 tokens a thread)
  int turn = 0;
  for_quads<VEC>(row, V, q0, q1, [&](const float4& x, int q) {
    const float v[4] = {x.x, x.y, x.z, x.w};
    uint32_t over = 0;  // bit e: above the window by its place, within the value of chi
    if ((v[0] <= v_hi && v[0] >= v_lo) || (v[1] <= v_hi && v[1] >= v_lo) || (v[2] <= v_hi && v[2] >= v_lo) ||
        (v[3] <= v_hi && v[3] >= v_lo)) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t cp = comp_of(v[e], q * 4 + e);
        if (v[e] <= v_hi && cp > chi) over |= 1u << e;
        if (cp <= chi && cp >= clo) {
          const int at = atomicAdd(n, 1);
          if (at < kList) list[at] = cp;
        }
      }
    }
    float w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool above = (v[e] > v_hi || (over >> e & 1)) && v[e] >= least;
      w[e] = above ? (v[e] == top ? 1.f : ex2(__fmul_rn(__fsub_rn(v[e], top), rate))) : 0.f;
    }
    part.add4(w);
    // (a weight of zero takes no part unless the bound is so low that any token may win)
    if (SCORE && fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])) >= start) {
      const uint4 ws = ph.block(static_cast<uint32_t>(q));
      if (race.may_win(w[0], ratio, ws.x) || race.may_win(w[1], ratio, ws.y) || race.may_win(w[2], ratio, ws.z) ||
          race.may_win(w[3], ratio, ws.w)) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if ((v[e] > v_hi || (over >> e & 1)) && v[e] >= least && race.may_win(w[e], ratio, word_of(ws, e))) {
            race.take(score_of(v[e], word_of(ws, e), p.temp), q * 4 + e);
            ratio = race.ratio_to(top, c);
          }
      }
    }
  }, [&] {
    if (SCORE && (turn & (turn + 1)) == 0) {  // a bound that the warp shares, after 1, 2, 4, ... turns
      race.warp_reduce();
      ratio = race.ratio_to(top, c);
    }
    ++turn;
  });
  mass = part.value();
}

// ---------------------------------------------------------------- the exact path
// The comp range of the tokens in value bins first .. last (the bin number
// falls as the key grows), at or above ulo: warps 0 and 1 find its ends.
template <typename F>
__device__ __forceinline__ void value_range(int first, int last, float top, F bin, uint64_t ulo, uint64_t* clo,
                                            uint64_t* chi) {
  const int warp = threadIdx.x >> 5;
  const uint32_t hi = key_of(top);
  if (warp == 0) {
    const uint32_t k = first_key(kKeyLowest, hi, [&](uint32_t key) { return bin(value_of(key)) <= last; });
    if ((threadIdx.x & 31) == 0) *clo = max(static_cast<uint64_t>(k) << 32, ulo);
  } else if (warp == 1) {
    // the first key past the bins, less one; none past them: up to `top`
    const uint32_t k = first_key(kKeyLowest, hi + 1, [&](uint32_t key) { return bin(value_of(key)) < first; });
    if ((threadIdx.x & 31) == 0) *chi = (static_cast<uint64_t>(k - 1) << 32) | 0xFFFFFFFFu;
  }
}

// One histogram over the tokens of [clo, chi] at or above ulo, and the bin
// where the criterion cuts: by_count, that of the top_k-th token; else the one
// in which the mass before a token reaches top_p of the total.  The first pass
// bins by value below `top`, the later ones by the place in [clo, chi].
// Narrows sh.clo / chi, adds to above_mass / above_n, sets in_n.
template <bool VEC>
__device__ void histogram_cut(SelShared& sh, const float* row, int V, const RowParam& p, float top, bool first,
                              uint64_t ulo, bool by_count) {
  const float c = mass_rate(p.temp), scale = __fdiv_rn(static_cast<float>(kBins) / kBinNats, p.temp);
  const uint64_t lo0 = sh.clo, hi0 = sh.chi, clo = max(lo0, ulo);
  const int shift = max(0, 64 - __clzll(static_cast<long long>(hi0 - lo0)) - 11);
  auto by_value = [&](float l) {
    const float d = l == top ? 0.f : __fmul_rn(__fsub_rn(top, l), scale);
    return d < static_cast<float>(kBins - 1) ? static_cast<int>(d) : kBins - 1;
  };
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kSelThreads) sh.h.cnt[i] = sh.h.lo[i] = sh.h.hi[i] = 0;
  __syncthreads();
  for_quads<VEC>(row, V, 0, (V + 3) / 4, [&](const float4& x, int q) {
    const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint64_t cp = comp_of(v[e], q * 4 + e);
      if (cp < clo || cp > hi0) continue;
      const int b = first ? by_value(v[e]) : static_cast<int>((hi0 - cp) >> shift);
      atomicAdd(&sh.h.cnt[b], 1u);
      const uint64_t w = fixed(weight(v[e], top, c));
      if (w) {
        const uint32_t wl = static_cast<uint32_t>(w), old = atomicAdd(&sh.h.lo[b], wl);
        const uint32_t up = static_cast<uint32_t>(w >> 32) + (old + wl < old ? 1u : 0u);
        if (up) atomicAdd(&sh.h.hi[b], up);
      }
    }
  }, [] {});
  __syncthreads();
  constexpr int PT = kBins / kSelThreads;
  const int b0 = threadIdx.x * PT, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto mass_of = [&](int b) { return sh.h.lo[b] + (static_cast<uint64_t>(sh.h.hi[b]) << 32); };
  uint32_t n = 0;
  uint64_t m = 0;
  for (int k = 0; k < PT; ++k) {
    n += sh.h.cnt[b0 + k];
    m += mass_of(b0 + k);
  }
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
  uint32_t an = sh.above_n + sn - n;
  uint64_t am = sh.above_mass + sm - m, total = sh.above_mass;
  for (int w = 0; w < kSelThreads / 32; ++w) {
    if (w < warp) {
      an += sh.redi[w];
      am += sh.redu[w];
    }
    total += sh.redu[w];
  }
  if (!first) total = sh.total_mass;  // the whole universe's, from the first pass
  const uint64_t want = share_of(p.top_p, total);
  __syncthreads();
  // the last non-empty bin before which the criterion still holds
  int cut = -1;
  uint32_t cut_n = 0, cut_in = 0;
  uint64_t cut_m = 0;
  for (int k = 0; k < PT; ++k) {
    const uint32_t bn = sh.h.cnt[b0 + k];
    if (bn && (by_count ? an < static_cast<uint32_t>(p.top_k) : an == 0 || am < want)) {
      cut = b0 + k;
      cut_n = an;
      cut_m = am;
      cut_in = bn;
    }
    an += bn;
    am += mass_of(b0 + k);
  }
  const int last = block_max(sh, cut);
  if (threadIdx.x == 0) {
    sh.total_mass = total;
    if (last < 0) sh.in_n = 0;  // an empty universe
  }
  if (cut == last && cut >= 0) {
    sh.above_n = cut_n;
    sh.above_mass = cut_m;
    sh.in_n = cut_in;
    if (first) {
      sh.flag = cut;  // its range of keys below
    } else {
      const uint64_t hi = hi0 - (static_cast<uint64_t>(cut) << shift), span = (1ull << shift) - 1;
      sh.chi = hi;
      sh.clo = max(max(lo0, hi > span ? hi - span : 0), ulo);
    }
  }
  __syncthreads();
  if (first && last >= 0) value_range(sh.flag, sh.flag, top, by_value, ulo, &sh.clo, &sh.chi);
  __syncthreads();
}

// A row by exact histograms, one CTA.
template <bool VEC>
__device__ __noinline__ void exact_row(SelShared& sh, const Out& o, int r, const RowParam& p, float top) {
  const float* row = o.logits + r * o.ld;
  const int V = o.V, quads = (V + 3) / 4;
  const bool has_k = p.top_k > 0, has_p = p.top_p < 1.f;
  const float least = min_p_least(p, top);
  uint64_t ulo = static_cast<uint64_t>(kKeyLowest) << 32;  // the universe: comp >= ulo
  auto narrow = [&](bool by_count) {  // each pass leaves at most 1 / 2048 of the range: six at most
    __syncthreads();
    if (threadIdx.x == 0) {
      sh.clo = ulo;
      sh.chi = ~0ull;
      sh.above_mass = 0;
      sh.above_n = 0;
      sh.in_n = 0;
    }
    __syncthreads();
    bool first = true;
    do {
      histogram_cut<VEC>(sh, row, V, p, top, first, ulo, by_count);
      first = false;
    } while (sh.in_n > kList);
  };
  Race race;
  auto collect = [&](float from, bool score) {  // the window's tokens, sorted and summed, and the mass above
    __syncthreads();
    if (threadIdx.x == 0) sh.n = 0;
    __syncthreads();
    uint64_t m;
    if (score) collect_quads<VEC, true>(row, V, 0, quads, p, top, from, sh.clo, sh.chi, sh.l.comp, &sh.n, race, m);
    else collect_quads<VEC, false>(row, V, 0, quads, p, top, from, sh.clo, sh.chi, sh.l.comp, &sh.n, race, m);
    const uint64_t above = block_sum(sh, m);
    const int n = min(sh.n, kList);
    sort_desc(sh.l.comp, n);
    prefix_mass(sh, n, top, p.temp, above);
    return above;
  };
  uint64_t z = 0;
  if (has_k) {
    narrow(true);
    if (has_p) {  // the top_k-th token and the mass down to it, then top-p within them
      const uint64_t above = collect(value_of(kKeyLowest), false);
      const int n = min(sh.n, kList), last = min(n, static_cast<int>(p.top_k - sh.above_n)) - 1;
      if (last >= 0) {
        ulo = sh.l.comp[last];
        z = sh.l.pre[last];
      } else {
        z = above;
      }
    }
  }
  if (has_p) {
    narrow(false);
    if (!has_k) z = sh.total_mass;
  } else if (!has_k) {  // min-p alone: every token is "above", nothing undecided
    __syncthreads();
    if (threadIdx.x == 0) {
      sh.clo = ulo;
      sh.chi = ulo - 1;
      sh.above_n = 0;
    }
    __syncthreads();
  }
  const uint64_t base = collect(least, true), want = share_of(p.top_p, z);
  const int n = min(sh.n, kList);
  int kept = 0;
  for (int j = threadIdx.x; j < n; j += kSelThreads) {
    const bool in_k = has_p || !has_k || sh.above_n + j < static_cast<uint32_t>(p.top_k);
    const bool in_p = !has_p || sh.above_n + j == 0 || (j == 0 ? base : sh.l.pre[j - 1]) < want;
    kept += in_k && in_p && value_of(static_cast<uint32_t>(sh.l.comp[j] >> 32)) >= least;
  }
  kept = block_sum(sh, kept);
  choose(sh, o, r, p, kept, race, kept > 0 ? sh.l.pre[kept - 1] : base, top, false);
}

// ---------------------------------------------------------------- select
// The race over the list's tokens of comp >= cut and value >= least.
__device__ void score_list(const SelShared& sh, const RowParam& p, int n, uint64_t cut, float least, Race& race) {
  const Philox ph(p);
  for (int j = threadIdx.x; j < n; j += kSelThreads) {
    const uint64_t cp = sh.l.comp[j];
    const float l = value_of(static_cast<uint32_t>(cp >> 32));
    if (cp < cut || l < least) continue;
    const int i = index_of(cp);
    race.take(score_of(l, word_of(ph.block(static_cast<uint32_t>(i) / 4), i & 3), p.temp), i);
  }
}

// The lowest comp among the list's tokens from `from` on before which weigh()'s
// sum is still below `want` (the first token's always): bins of value, their
// weights as integers, then the cut's bin token by token.  False: that bin is
// too large (ties).  bottom: no listed token's value is below it.
template <typename W>
__device__ __forceinline__ bool list_cut(SelShared& sh, int n, float top, float bottom, uint64_t from, uint64_t want,
                                         W weigh, uint64_t* cut) {
  auto& b = sh.l.b;
  const float scale = __fdiv_rn(static_cast<float>(kListBins - 1), __fsub_rn(top, bottom));
  auto bin = [&](uint64_t cp) {
    const float l = value_of(static_cast<uint32_t>(cp >> 32));
    const float d = l == top ? 0.f : __fmul_rn(__fsub_rn(top, l), scale);
    return d < static_cast<float>(kListBins - 1) ? static_cast<int>(d) : kListBins - 1;
  };
  __syncthreads();
  for (int i = threadIdx.x; i < kListBins; i += kSelThreads) b.cnt[i] = b.lo[i] = b.hi[i] = 0;
  if (threadIdx.x == 0) sh.in_n = 0;
  __syncthreads();
  for (int j = threadIdx.x; j < n; j += kSelThreads) {
    if (sh.l.comp[j] < from) continue;
    const uint64_t w = weigh(sh.l.comp[j]);
    const int i = bin(sh.l.comp[j]);
    const uint32_t wl = static_cast<uint32_t>(w), old = atomicAdd(&b.lo[i], wl);
    const uint32_t up = static_cast<uint32_t>(w >> 32) + (old + wl < old ? 1u : 0u);
    if (up) atomicAdd(&b.hi[i], up);
    atomicAdd(&b.cnt[i], 1u);
  }
  __syncthreads();
  constexpr int PT = kListBins / kSelThreads;
  const int b0 = threadIdx.x * PT, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t m = 0;
#pragma unroll
  for (int k = 0; k < PT; ++k) m += b.lo[b0 + k] + (static_cast<uint64_t>(b.hi[b0 + k]) << 32);
  uint64_t am = m;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const uint64_t x = __shfl_up_sync(0xffffffffu, am, s);
    if (lane >= s) am += x;
  }
  if (lane == 31) sh.redu[warp] = am;
  __syncthreads();
  am -= m;
  for (int w = 0; w < warp; ++w) am += sh.redu[w];
  int last = -1;  // the last bin before which the sum is below `want` (the first bin with a token at least)
  uint64_t last_m = 0;
#pragma unroll
  for (int k = 0; k < PT; ++k) {
    if (b.cnt[b0 + k] && (am == 0 || am < want)) {
      last = b0 + k;
      last_m = am;
    }
    am += b.lo[b0 + k] + (static_cast<uint64_t>(b.hi[b0 + k]) << 32);
  }
  const int cut_bin = block_max(sh, last);
  if (last == cut_bin) sh.above_mass = last_m;
  __syncthreads();
  const uint64_t before = sh.above_mass;
  for (int j = threadIdx.x; j < n; j += kSelThreads)
    if (sh.l.comp[j] >= from && bin(sh.l.comp[j]) == cut_bin) {
      const uint32_t at = atomicAdd(&sh.in_n, 1u);
      if (at < kCutList) b.cut[at] = sh.l.comp[j];
    }
  __syncthreads();
  const int in = static_cast<int>(sh.in_n);
  if (in > kCutList) return false;
  // a token of the bin is kept if the sum before it (over those of larger comp) stays below `want`
  uint64_t lowest = ~0ull;
  for (int j = threadIdx.x; j < in; j += kSelThreads) {
    const uint64_t mine = b.cut[j];
    uint64_t ahead = before;
    for (int k = 0; k < in; ++k)
      if (b.cut[k] > mine) ahead += weigh(b.cut[k]);
    if ((ahead < want || ahead == 0) && mine < lowest) lowest = mine;
  }
  *cut = block_reduce(lowest, sh.redu, [](uint64_t x, uint64_t y) { return x < y ? x : y; });
  return true;
}

// A row by its unsorted list of n tokens, which are all tokens at or above
// `bottom` (complete: all there are): true if that decides it.  An undecided row
// of which every listed token is kept leaves the best of their scores in `best`
// (bound: asked for).
__device__ __noinline__ bool cut_unsorted(SelShared& sh, const Out& o, int r, const RowParam& p, int n, float top,
                                          float bottom, uint64_t z, bool complete, bool bound, Race& best) {
  const bool has_p = p.top_p < 1.f, has_k = p.top_k > 0, k_listed = has_k && p.top_k <= n;
  if (has_k && has_p && !k_listed && !complete) return false;  // top-p's share is of the top-k's mass
  const float least = min_p_least(p, top);
  const float c = mass_rate(p.temp);
  auto mass_of = [&](uint64_t cp) { return mass_at(cp, top, c); };
  int below = 0;  // listed tokens that min-p drops
  float low = top;
  for (int j = threadIdx.x; j < n; j += kSelThreads) {
    const float l = value_of(static_cast<uint32_t>(sh.l.comp[j] >> 32));
    below += l < least;
    low = fminf(low, l);
  }
  if (complete)  // (`bottom` is then no logit's, but the lowest finite value)
    bottom = value_of(block_reduce(key_of(low), reinterpret_cast<uint32_t*>(sh.redi),
                                   [](uint32_t x, uint32_t y) { return min(x, y); }));
  below = block_sum(sh, below);
  uint64_t cut = 0;  // the lowest kept comp
  if (k_listed && !list_cut(sh, n, top, bottom, 0, p.top_k, [](uint64_t) { return 1ull; }, &cut)) return false;
  bool decided = complete || below > 0 || k_listed;
  if (has_p) {
    uint64_t mass = 0;
    for (int j = threadIdx.x; j < n; j += kSelThreads)
      if (sh.l.comp[j] >= cut) mass += mass_of(sh.l.comp[j]);
    mass = block_sum(sh, mass);
    const uint64_t want = share_of(p.top_p, has_k ? mass : z);
    if (mass >= want) {
      decided = true;
      if (!list_cut(sh, n, top, bottom, cut, want, mass_of, &cut)) return false;
    }
  }
  if (!decided) {
    if (bound) {
      score_list(sh, p, n, 0, least, best);
      block_best(sh, best);
    }
    return false;
  }
  uint64_t kept = 0;
  Race race;
  for (int j = threadIdx.x; j < n; j += kSelThreads) {
    const uint64_t cp = sh.l.comp[j];
    if (cp >= cut && value_of(static_cast<uint32_t>(cp >> 32)) >= least) kept += mass_of(cp);
  }
  kept = block_sum(sh, kept);
  score_list(sh, p, n, cut, least, race);
  choose(sh, o, r, p, 0, race, kept, top, false);
  return true;
}

// wide_next: the count and collect kernels follow, and take rows that the
// lists do not decide.  Bound by a row's chain of small steps (segment maxima,
// gather, cut, race): 12 us for one row, 23 us for 256 of mixed settings, two to
// an SM; sorting every list took 17 and 29 us.
template <bool VEC>
__global__ void __launch_bounds__(kSelThreads) filter_select_kernel(Out o, Space sp, bool wide_next) {
  __shared__ SelShared sh;
  extern __shared__ float seg_max[];                     // [nseg]
  int* seg_n = reinterpret_cast<int*>(seg_max + o.nseg);  // [nseg] list entries
  int* seg_off = seg_n + o.nseg;                          // [nseg] where a list starts among those taken
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x, lane = threadIdx.x & 31;
  const RowParam p = sp.params[r];
  const int mode = row_mode(p);
  const SegOut* segs = sp.segs + static_cast<size_t>(r) * o.nseg;
  float top = -INFINITY;
  uint32_t floor = kKeyLowest;  // every logit from here on is listed
  Race race;
  for (int i = threadIdx.x; i < o.nseg; i += kSelThreads) {
    const SegOut s = segs[i];
    seg_max[i] = s.max;
    seg_n[i] = s.count;
    top = fmaxf(top, s.max);
    floor = max(floor, s.thr);
    if (better(s.best, s.best_i, race.best, race.best_i)) {
      race.best = s.best;
      race.best_i = s.best_i;
    }
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    floor = max(floor, __shfl_xor_sync(0xffffffffu, floor, s));
  }
  if (lane == 0) {
    sh.redf[threadIdx.x >> 5] = top;
    sh.redi[threadIdx.x >> 5] = static_cast<int>(floor);
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    top = fmaxf(top, sh.redf[w]);
    floor = max(floor, static_cast<uint32_t>(sh.redi[w]));
  }
  uint64_t z = 0;
  if (needs_mass(p)) {
    const float c = mass_rate(p.temp);
    for (int i = threadIdx.x; i < o.nseg; i += kSelThreads)
      z += fixed(__fmul_rn(segs[i].sum, weight(seg_max[i], top, c)));
    z = block_sum(sh, z);
  }
  if (mode != ROW_FILTER || top == -INFINITY) {  // (without any finite logit the filters do not matter)
    __syncthreads();
    choose(sh, o, r, p, 0, race, z, top, mode != ROW_FREE || top == -INFINITY);
    return;
  }
  const bool all = floor <= kKeyLowest;  // the lists hold every finite logit
  Race listed;  // the best of the listed tokens, where they are all kept
  // Level 0: as many candidates as there are large segment maxima (at least the
  // first `want` tokens are among those at or above the want-th largest).  Level
  // 1: every listed one.  Rows with a top-k take the few first; the others all
  // (61 wide rows 22 -> 16 us), and the few only where those are too many.
  for (int turn = 0; turn < 2; ++turn) {
    const int level = p.top_k > 0 ? turn : 1 - turn;
    const bool last = turn == 1 || p.top_k == 0;  // what is undecided then goes on to the wide kernels
    uint32_t from = floor;
    if (level == 0) {
      const int want = min(p.top_k > 0 ? p.top_k : 48, o.nseg);
      uint32_t mine = 0;  // the want-th largest segment maximum's key
      for (int i = threadIdx.x; i < o.nseg; i += kSelThreads) {
        int above = 0;
        const float m = seg_max[i];
#pragma unroll 8
        for (int j = 0; j < o.nseg; ++j) above += seg_max[j] > m || (seg_max[j] == m && j < i);
        if (above == want - 1) mine = key_of(m);
      }
      from = max(block_reduce(mine, reinterpret_cast<uint32_t*>(sh.redi),
                              [](uint32_t x, uint32_t y) { return max(x, y); }),
                 floor);
      if (from == floor) continue;
    }
    __syncthreads();
    if (threadIdx.x == 0) sh.n = 0;
    __syncthreads();
    // the qualifying segments' lists end to end: entry e is in the last segment that starts at or before it
    const int per = (o.nseg + kSelThreads - 1) / kSelThreads, s0 = threadIdx.x * per, s1 = min(o.nseg, s0 + per);
    int mine = 0;
    for (int i = s0; i < s1; ++i) mine += key_of(seg_max[i]) >= from ? seg_n[i] : 0;
    int start = mine;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, start, s);
      if (lane >= s) start += x;
    }
    if (lane == 31) sh.redi[threadIdx.x >> 5] = start;
    __syncthreads();
    start -= mine;
    int entries = 0;
#pragma unroll
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < static_cast<int>(threadIdx.x >> 5)) start += sh.redi[w];
      entries += sh.redi[w];
    }
    for (int i = s0; i < s1; ++i) {
      seg_off[i] = start;
      start += key_of(seg_max[i]) >= from ? seg_n[i] : 0;
    }
    __syncthreads();
    constexpr int kAhead = 4;
    for (int e0 = threadIdx.x; e0 < entries; e0 += kAhead * kSelThreads) {
      uint64_t cp[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int e = e0 + u * kSelThreads;
        if (e >= entries) continue;
        int a = 0, b = o.nseg - 1;
        while (a < b) {
          const int mid = (a + b + 1) >> 1;
          if (seg_off[mid] <= e) a = mid;
          else b = mid - 1;
        }
        cp[u] = sp.lists[(static_cast<size_t>(r) * o.nseg + a) * kSegCap + (e - seg_off[a])];
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (e0 + u * kSelThreads < entries && static_cast<uint32_t>(cp[u] >> 32) >= from) {
          const int at = atomicAdd(&sh.n, 1);
          if (at < kList) sh.l.comp[at] = cp[u];
        }
    }
    __syncthreads();
    const int n = sh.n;
    if (n > kList || n == 0) continue;  // too many candidates, or none listed (ties)
    const bool complete = all && from == floor;
    if (n > kFew) {  // no order is needed but at the cut
      if (cut_unsorted(sh, o, r, p, n, top, value_of(from), z, complete, last && wide_next, listed)) return;
      if (p.top_k == 0) break;
      continue;
    }
    sort_few(sh.l.comp, n);
    prefix_mass(sh, n, top, p.temp, 0);
    const int lim = p.top_k > 0 ? min(p.top_k, n) : n;
    const bool k_known = complete || p.top_k <= n;  // with top_k on: the list holds all of its tokens
    const bool has_p = p.top_p < 1.f;
    if (p.top_k > 0 && has_p && !k_known) continue;
    const uint64_t share = has_p ? share_of(p.top_p, p.top_k > 0 ? sh.l.pre[lim - 1] : z) : 0;
    int kept = 0;
    for (int j = threadIdx.x; j < lim; j += kSelThreads) {
      const float l = value_of(static_cast<uint32_t>(sh.l.comp[j] >> 32));
      kept += (!has_p || j == 0 || sh.l.pre[j - 1] < share) && min_p_keeps(l, top, p.temp, p.log_min_p);
    }
    kept = block_sum(sh, kept);
    const bool decided = complete || kept < n || (p.top_k > 0 && p.top_k <= n) || (has_p && sh.l.pre[lim - 1] >= share);
    if (!decided) {
      if (last && wide_next) {  // every listed token is kept
        score_list(sh, p, n, 0, -INFINITY, listed);
        block_best(sh, listed);
      }
      if (p.top_k == 0) break;
      continue;
    }
    choose(sh, o, r, p, kept, Race(), kept > 0 ? sh.l.pre[kept - 1] : 0, top, false);
    return;
  }
  if (!wide_next || (p.top_k > 0 && p.top_p < 1.f)) {
    exact_row<VEC>(sh, o, r, p, top);
    return;
  }
  for (int i = threadIdx.x; i < kCountBins; i += kSelThreads) sp.count[static_cast<size_t>(r) * kCountBins + i] = 0;
  // The bins of `count` reach from the largest logit down to the lowest of 4096
  // spread over the row (lower ones share the last bin), kBinNats T at most: a
  // bin of a flat row then holds few enough tokens to list.
  float low = top;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float4 x = load4<VEC>(o.logits + r * o.ld, (u * kSelThreads + static_cast<int>(threadIdx.x)) *
                                                         ((o.V + 3) / 4) / (4 * kSelThreads) * 4, o.V);
    const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (v[e] >= value_of(kKeyLowest)) low = fminf(low, v[e]);
  }
  low = value_of(block_reduce(key_of(low), reinterpret_cast<uint32_t*>(sh.redi),
                              [](uint32_t x, uint32_t y) { return min(x, y); }));
  if (threadIdx.x < 32) {
    WideState w{};
    const float most = __fmul_rn(kBinNats, p.temp), range = __fsub_rn(top, low);
    w.range = range > 0.f ? fminf(range, most) : most;
    w.z = z;
    w.top = top;
    w.least = min_p_least(p, top);
    if (lane != 0) return;
    w.bound = listed.best;
    w.clo = static_cast<uint64_t>(kKeyLowest) << 32;  // min-p alone: an empty window below every token
    w.chi = w.clo - 1;
    sp.wide[r] = w;
    sp.wide_rows[atomicAdd(sp.n_wide, 1)] = r;  // in any order: rows do not depend on one another
  }
}

// ---------------------------------------------------------------- wide rows
// 61 rows of 262144 (64 MB, in L2 after the scan): count 44 us, bound by its
// shared-memory atomics; collect 63 to 70 us, bound by issue (Philox and the
// race's bound, 70 warp instructions per 32 tokens).  A few wide rows among 256
// take 20 us each, the chain of one part and of the row's last CTA.
// Whether this CTA is the last of a row's `total` to arrive; what the others
// wrote before arriving is then visible to it.
__device__ __forceinline__ bool last_arrival(uint32_t* arrived, int total, int* flag) {
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) *flag = atomicAdd(arrived, 1u) == static_cast<uint32_t>(total) - 1;
  __syncthreads();
  const bool last = *flag != 0;
  if (last) __threadfence();
  return last;
}

// The CTA's next work item, in the order the CTAs ask.
__device__ __forceinline__ int next_item(int* counter, int* slot) {
  __syncthreads();
  if (threadIdx.x == 0) *slot = atomicAdd(counter, 1);
  __syncthreads();
  return *slot;
}

// A wide row's parts, one work item each: as many as the grid has CTAs for, in
// the fewest whole rounds that leave a row 8 (so that no more than one CTA in
// nine idles in the last), and none below kChunk tokens.
struct Parts {
  int n, quads;  // parts of a row; quads of a part
  __device__ __forceinline__ Parts(int n_wide, int V) {
    const int all = (V + 3) / 4, grid = static_cast<int>(gridDim.x);
    int most = 1;  // (no wide row: no items)
    if (n_wide > 0) most = max(1, (8 * n_wide + grid - 1) / grid * grid / n_wide);
    n = min(most, (V + kChunk - 1) / kChunk);
    quads = ((all + n - 1) / n + 7) / 8 * 8;
    n = (all + quads - 1) / quads;
  }
};

// A token's place in its row's value bins: bin << 5 | 32nd of the bin, to the
// nearest (adding 2^23 rounds to a whole number in the low bits, where a
// conversion would take the slow unit).
__device__ __forceinline__ uint32_t value_place(float l, float top, float scale32) {
  const float d = fminf(__fmul_rn(__fsub_rn(top, l), scale32), static_cast<float>((kCountBins - 1) * 32));
  return __float_as_uint(__fadd_rn(l == top ? 0.f : d, 8388608.f)) & 0x7FFFFFu;
}

// The estimate of a bin's mass from its tokens' mean place is off by the
// rounding of the places (half a 32nd of a bin's 0.6 %, at most 9e-5 of the
// bin's mass and less for values in no order) and by the spread inside a bin
// (2e-6): the window takes 1 / kSlack of the whole mass to either side, and
// `collect` checks the sums themselves.
constexpr int kSlack = 10000;

template <bool VEC>
__global__ void __launch_bounds__(kSelThreads, 3) filter_count_kernel(Out o, Space sp) {
  __shared__ SelShared sh;
  pdl_wait();
  pdl_trigger();
  const int n_wide = *reinterpret_cast<volatile int*>(sp.n_wide);
  const Parts ps(n_wide, o.V);
  const int parts = ps.n, items = n_wide * parts;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int item; (item = next_item(sp.n_wide + 1, &sh.n)) < items;) {
    const int r = sp.wide_rows[item / parts], part = item % parts;
    const RowParam p = sp.params[r];
    const bool by_count = p.top_k > 0;
    if (!by_count && p.top_p >= 1.f) continue;  // min-p alone needs no window
    WideState& st = sp.wide[r];
    const float top = st.top, scale32 = __fdiv_rn(32.f * kCountBins, st.range);
    const float low = value_of(kKeyLowest);
    constexpr int PT = kCountBins / kSelThreads;
    uint32_t bn[PT], bp[PT];  // tokens and places of bins threadIdx.x + k * kSelThreads
#pragma unroll
    for (int k = 0; k < PT; ++k) bn[k] = bp[k] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PT; ++k) sh.count[threadIdx.x + k * kSelThreads] = 0;
    const int end = min((o.V + 3) / 4, (part + 1) * ps.quads);
    for (int q0 = part * ps.quads; q0 < end; q0 += kCountTurn / 4) {
      __syncthreads();
      // tokens in the upper 14 bits, the sum of their 32nds in the lower 18: no
      // bin of 8192 tokens carries over (8192 * 31 < 2^18, and 8192 < 2^14)
      static_assert(kCountTurn * 31 < (1 << 18) && kCountTurn < (1 << 14), "packed counters");
      for_quads<VEC>(o.logits + r * o.ld, o.V, q0, min(end, q0 + kCountTurn / 4), [&](const float4& x, int) {
        const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (v[e] >= low) {
            const uint32_t at = value_place(v[e], top, scale32);
            atomicAdd(&sh.count[at >> 5], (at & 31) | (1u << 18));
          }
      }, [] {});
      __syncthreads();
#pragma unroll
      for (int k = 0; k < PT; ++k) {
        const uint32_t h = sh.count[threadIdx.x + k * kSelThreads];
        sh.count[threadIdx.x + k * kSelThreads] = 0;
        bn[k] += h >> 18;
        bp[k] += h & 0x3FFFF;
      }
    }
    unsigned long long* count = sp.count + static_cast<size_t>(r) * kCountBins;
#pragma unroll
    for (int k = 0; k < PT; ++k)  // (V <= 2^21: the places' sum stays below 2^26)
      if (bn[k]) atomicAdd(&count[threadIdx.x + k * kSelThreads], static_cast<unsigned long long>(bn[k]) << 32 | bp[k]);
    if (!last_arrival(&st.arrived[0], parts, &sh.flag)) continue;
    // ---- the window
    const int b0 = threadIdx.x * PT;
    const float step = __fdiv_rn(st.range, __fmul_rn(p.temp, static_cast<float>(kCountBins)));  // nats of a bin
    uint64_t bm[PT];
    uint32_t n = 0;
    uint64_t m = 0;
#pragma unroll
    for (int k = 0; k < PT; ++k) {
      const unsigned long long both = __ldcg(&count[b0 + k]);
      bn[k] = static_cast<uint32_t>(both >> 32);
      const float mean = __fdiv_rn(static_cast<float>(static_cast<uint32_t>(both)), 32.f * fmaxf(static_cast<float>(bn[k]), 1.f));
      bm[k] = fixed(__fmul_rn(static_cast<float>(bn[k]), ex2(__fmul_rn(-step * kLog2e, __fadd_rn(static_cast<float>(b0 + k),
                                                                                    mean)))));
      n += bn[k];
      m += bm[k];
    }
    uint32_t sn = n;
    uint64_t sm = m;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const uint32_t xn = __shfl_up_sync(0xffffffffu, sn, s);
      const uint64_t xm = __shfl_up_sync(0xffffffffu, sm, s);
      if (lane >= s) {
        sn += xn;
        sm += xm;
      }
    }
    if (lane == 31) {
      sh.redi[warp] = static_cast<int>(sn);
      sh.redu[warp] = sm;
    }
    __syncthreads();
    uint32_t an = sn - n;
    uint64_t am = sm - m;
    for (int w = 0; w < warp; ++w) {
      an += sh.redi[w];
      am += sh.redu[w];
    }
    const uint64_t z = st.z, want = share_of(p.top_p, z), slack = z / kSlack;
    int lo = kCountBins, hi = -1;  // the window's first and last bin
    uint32_t lo_n = 0, hi_n = 0;   // tokens above the first, tokens up to the last
#pragma unroll
    for (int k = 0; k < PT; ++k) {
      if (bn[k]) {
        const bool enters = by_count ? an + bn[k] >= static_cast<uint32_t>(p.top_k) : am + bm[k] + slack > want;
        const bool holds = by_count ? an < static_cast<uint32_t>(p.top_k) : an == 0 || am < want + slack;
        if (enters && lo == kCountBins) {
          lo = b0 + k;
          lo_n = an;
        }
        if (holds) {
          hi = b0 + k;
          hi_n = an + bn[k];
        }
      }
      an += bn[k];
      am += bm[k];
    }
    __syncthreads();
    const int last = block_max(sh, hi);
    const int first = min(-block_max(sh, -lo), last);
    if (threadIdx.x == 0) sh.above_n = sh.in_n = 0xFFFFFFFFu;
    __syncthreads();
    if (last >= 0 && lo == first) sh.above_n = lo_n;
    if (last >= 0 && hi == last) sh.in_n = hi_n;
    __syncthreads();
    const bool found = sh.above_n <= sh.in_n && sh.in_n != 0xFFFFFFFFu;
    if (threadIdx.x == 0) {
      st.above_n = sh.above_n;
      st.in_n = found ? sh.in_n - sh.above_n : 0xFFFFFFFFu;
    }
    if (found)
      value_range(first, last, top, [&](float l) { return static_cast<int>(value_place(l, top, scale32) >> 5); }, 0, &st.clo, &st.chi);
  }
}

template <bool VEC>
__global__ void __launch_bounds__(kSelThreads, 4) filter_collect_kernel(Out o, Space sp) {
  __shared__ SelShared sh;
  pdl_wait();
  pdl_trigger();
  const int n_wide = *reinterpret_cast<volatile int*>(sp.n_wide);
  const Parts ps(n_wide, o.V);
  const int parts = ps.n, items = n_wide * parts;
  for (int item; (item = next_item(sp.n_wide + 2, &sh.n)) < items;) {
    const int r = sp.wide_rows[item / parts], part = item % parts;
    const RowParam p = sp.params[r];
    WideState& st = sp.wide[r];
    const bool has_k = p.top_k > 0, has_p = p.top_p < 1.f;
    const float top = st.top, least = st.least;
    if ((has_k || has_p) && st.in_n > kList) {  // no window
      if (part == 0) exact_row<VEC>(sh, o, r, p, top);
      continue;
    }
    Race race;
    race.best = st.bound;  // with no token: any that reaches it takes over
    race.set_bound();
    uint64_t mass;
    uint64_t* window = sp.window + static_cast<size_t>(r) * kList;
    const int q0 = part * ps.quads;
    if (threadIdx.x == 0) sh.listed = 0;
    __syncthreads();
    collect_quads<VEC, true>(o.logits + r * o.ld, o.V, q0, min((o.V + 3) / 4, q0 + ps.quads), p, top, least, st.clo,
                             st.chi, sh.l.comp, &sh.listed, race, mass);
    __syncthreads();
    if (const int mine = min(sh.listed, kList); mine > 0) {  // to the row's list, in one piece
      __syncthreads();
      if (threadIdx.x == 0) sh.listed = atomicAdd(&st.n, mine);
      __syncthreads();
      const int at = sh.listed;
      for (int j = threadIdx.x; j < mine && at + j < kList; j += kSelThreads) window[at + j] = sh.l.comp[j];
    }
    const uint64_t sum = block_sum(sh, mass);
    block_best(sh, race);
    ChunkOut* chunks = sp.chunks + static_cast<size_t>(r) * o.nchunk;
    if (threadIdx.x == 0) chunks[part] = ChunkOut{sum, race.best, race.best_i};
    if (!last_arrival(&st.arrived[1], parts, &sh.flag)) continue;
    // ---- the choice
    uint64_t base = 0;
    Race best;
    for (int k = threadIdx.x; k < parts; k += kSelThreads) {
      const ChunkOut* co = chunks + k;
      base += __ldcg(reinterpret_cast<const unsigned long long*>(&co->mass));
      const float b = __ldcg(&co->best);
      const int bi = __ldcg(&co->best_i);
      if (better(b, bi, best.best, best.best_i)) {
        best.best = b;
        best.best_i = bi;
      }
    }
    base = block_sum(sh, base);
    const int n = min(__ldcg(&st.n), kList);
    for (int j = threadIdx.x; j < n; j += kSelThreads) sh.l.comp[j] = __ldcg(reinterpret_cast<const unsigned long long*>(window) + j);
    __syncthreads();
    sort_desc(sh.l.comp, n);
    prefix_mass(sh, n, top, p.temp, base);
    const uint64_t want = share_of(p.top_p, st.z);
    // Does the window hold the cut?  (Where min-p starts above it, min-p cuts and not top-p.)
    const bool min_cuts = least > value_of(static_cast<uint32_t>(st.chi >> 32));
    if (has_p && !min_cuts && !((st.above_n == 0 || base < want) && n > 0 && sh.l.pre[n - 1] >= want)) {
      exact_row<VEC>(sh, o, r, p, top);
      continue;
    }
    int kept = 0;
    for (int j = threadIdx.x; j < n; j += kSelThreads) {
      const bool in_k = !has_k || st.above_n + j < static_cast<uint32_t>(p.top_k);
      const bool in_p = !has_p || st.above_n + j == 0 || (j == 0 ? base : sh.l.pre[j - 1]) < want;
      kept += in_k && in_p && value_of(static_cast<uint32_t>(sh.l.comp[j] >> 32)) >= least;
    }
    kept = block_sum(sh, kept);
    choose(sh, o, r, p, kept, best, kept > 0 ? sh.l.pre[kept - 1] : base, top, false);
  }
}

// ---------------------------------------------------------------- host
int sm_count_filter() {
  static int n = 0;
  if (!n) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
  }
  return n;
}

void row_param(const SampleFilterArgs& a, int r, RowParam* p) {
  const vd_sampler& s = a.samplers[r];
  p->seed = s.seed;
  p->step = s.step;
  p->temp = s.temperature;
  p->top_p = 1.f;
  p->log_min_p = -INFINITY;
  p->top_k = 0;
  if (a.filters) {
    const vd_filter& f = a.filters[r];
    p->top_k = f.top_k > 0 && f.top_k < a.V ? f.top_k : 0;
    p->top_p = f.top_p;
    p->log_min_p = f.min_p > 0.f ? static_cast<float>(log(static_cast<double>(f.min_p))) : -INFINITY;
  }
}

// Rows whose top_k is at most this are decided by their lists unless the
// logits are adversarial (the lists hold about 1000 tokens of logits in no
// order): a call of such rows alone does without the wide kernels.
constexpr int kNarrowK = 256;

template <int N>
int launch_scan(const SampleFilterArgs& a, const Space& sp, int nseg, int r0, int rows, bool vec, bool* wide,
                cudaStream_t s) {
  // Unfiltered rows (four times a filtered row's work) first, then those whose
  // mass is asked for: every warp's turns then cost about the same.
  RowParams<N> params;
  RowParam given[N];
  int at[3] = {0, 0, 0};
  auto kind = [](const RowParam& p) { return row_mode(p) == ROW_FREE ? 0 : needs_mass(p) ? 1 : 2; };
  for (int i = 0; i < rows; ++i) {
    row_param(a, r0 + i, &given[i]);
    const RowParam& p = given[i];
    *wide |= p.temp > 0.f && !(p.top_k > 0 && p.top_k <= kNarrowK) &&
             (p.top_k > 0 || p.top_p < 1.f || p.log_min_p > -INFINITY);
    ++at[kind(p)];
  }
  at[2] = at[0] + at[1];
  at[1] = at[0];
  at[0] = 0;
  for (int i = 0; i < rows; ++i) {
    const int k = at[kind(given[i])]++;
    params.r[k] = given[i];
    params.row[k] = static_cast<short>(i);
  }
  for (int i = rows; i < N; ++i) {
    params.r[i] = RowParam{};
    params.row[i] = 0;
  }
  // 8 groups list about 22 logits of a segment, 4 about 8, 2 about 3: a row's lists hold 1000 to 3000 in all, and
  // those from its largest threshold on fit a CTA's list
  const int groups = nseg <= 128 ? 8 : nseg <= 384 ? 4 : 2;
  VD_CUDA_TRY(launch_k(vec ? filter_scan_kernel<N, true> : filter_scan_kernel<N, false>,
                       dim3(std::min((rows * nseg + kScanThreads / 32 - 1) / (kScanThreads / 32),
                                     kScanCtas * sm_count_filter())),
                       dim3(kScanThreads), 0, s, params, a.logits, a.V, a.ld, nseg, groups, r0 == 0, sp, r0, rows));
  return VD_OK;
}

template <bool VEC>
int launch_decide(const Out& o, const Space& sp, int R, bool wide, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(o.nseg) * 12;
  if (smem + sizeof(SelShared) > 48 * 1024)  // the most that any launch takes: another thread's may come in between
    VD_CUDA_TRY(cudaFuncSetAttribute(filter_select_kernel<VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (kFilterMaxVocab + kSeg - 1) / kSeg * 12));
  VD_CUDA_TRY(launch_k(filter_select_kernel<VEC>, dim3(R), dim3(kSelThreads), smem, s, o, sp, wide));
  if (!wide) return VD_OK;
  const long long most = static_cast<long long>(R) * o.nchunk, n_sm = sm_count_filter();
  VD_CUDA_TRY(launch_k(filter_count_kernel<VEC>, dim3(static_cast<unsigned>(std::min(most, 3 * n_sm))), dim3(kSelThreads),
                       0, s, o, sp));
  VD_CUDA_TRY(launch_k(filter_collect_kernel<VEC>, dim3(static_cast<unsigned>(std::min(most, 4 * n_sm))),
                       dim3(kSelThreads), 0, s, o, sp));
  return VD_OK;
}

int segments(int V) { return (V + kSeg - 1) / kSeg; }
int chunks_of(int V) { return (V + kChunk - 1) / kChunk; }

}  // namespace

size_t sample_filter_workspace(int R, int V) {
  Space sp;
  return space_of(&sp, nullptr, R, segments(V), chunks_of(V));
}

int launch_sample_filter(const SampleFilterArgs& a, cudaStream_t s, int* launched) {
  Out o{a.logits, a.ld, a.V, segments(a.V), chunks_of(a.V), a.tokens, a.logprobs};
  Space sp;
  space_of(&sp, a.workspace, a.R, o.nseg, o.nchunk);
  const bool vec = (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0 && a.ld % 4 == 0;
  bool wide = false;
  int rc = VD_OK;
  const int launches = (a.R + kScanRows - 1) / kScanRows, each = (a.R + launches - 1) / launches;
  for (int r0 = 0; r0 < a.R; r0 += each) {
    const int rows = std::min(each, a.R - r0);
    rc = rows <= 16 ? launch_scan<16>(a, sp, o.nseg, r0, rows, vec, &wide, s)
         : rows <= 120 ? launch_scan<120>(a, sp, o.nseg, r0, rows, vec, &wide, s)
                       : launch_scan<kScanRows>(a, sp, o.nseg, r0, rows, vec, &wide, s);
    if (rc) return rc;
  }
  if (launched) *launched = launches + (wide ? 3 : 1);
  return vec ? launch_decide<true>(o, sp, a.R, wide, s) : launch_decide<false>(o, sp, a.R, wide, s);
}

}  // namespace vd
