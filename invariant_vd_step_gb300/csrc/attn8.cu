// Attention over the 8-bit KV cache: mma.sync kernel.
//
// Rows and splits are those of attention.cu: for request b and KV head g the
// (token, query head of the group) pairs, token-major, in blocks of 16, and
// splits of 512 keys.  A split is four chunks of 128 keys (eight pages), one per
// warp.  What a row sees of a page i: its 8-bit version if i < own = floor(p /
// 16), its bf16 version if i = own, nothing beyond.
//
// Per chunk and row, with codes c, K scale k, V scale v of each page and
// everything else float32 unless stated; 0 marks what the chunks of the split before
// this one left (S = -inf at the first):
//   s_j = (q c_j) k scale                (the product in fp16, exact operands)
//   S   = max(S0, max_j s_j),   r = max_j (s_j + log2 v_j) - S
//   u   = max(log2 v - r, -90),  p_j = 2^(s_j - (S - u)),   w_j = p_j 2^-u = 2^(s_j - S)
//   l   = l 2^(S0 - S) + sum_j w_j
//   O   = O 2^(S0 - S + r0 - r) + sum_j fp16(p_j) c_j
// so O 2^r / l is the softmax's mean of the values, and a split's partial is (S, l, O
// 2^r), the last two times 2^-24.  The V scale rides in the exponent and the codes enter
// the product as they are; r makes the largest p of the row 1, and fp16 rounds p by
// 2^-12 of itself or 2^-25, where bf16 would be off by 2^-9.  (The kernels of the 16-bit
// cache hold p as two bf16 terms, 2^-17, at twice the products: here the codes are 2^-8
// of a page's largest or 2^-4 of themselves off, and the output is rounded by 2^-9, so that
// outputs are 0.0017 off the exact ones of these codes either way.)  S and l know nothing of V:
// with p relative to the largest alone, keys whose V is 2^126 below the largest, or 0,
// would leave the denominator.  With the bound -90 of u (below it nothing of p is left
// in fp16) each weight of 2^-36 of the largest and more is in l whatever the V, and
// where no V is that far apart all down to 2^-126.  The row's own page takes part with a
// scale per token, a power of two that makes its bf16 values exact in fp16 (kv8.cuh).
//
// Order: the pages of a chunk ascending, the own page last.  Keys 2t + e and 2t +
// 8 + e of each page go to the partial sum l_(t, e) of eight, t < 4, e < 2, of
// the half of the chunk (four pages) that they are in; the half's l is the sum
// over t, as (0 + 1) + (2 + 3), of l_(t, 0) + l_(t, 1), and the halves are added at
// the end of the split.  The four chunks of a split run side by side, one per
// warp, share their maxima before they take their weights, and are folded left to
// right (one fma per value); the merge kernel folds the splits.  A masked key has
// the weight 0 and adds +0 to every sum.  None of it depends on the batch, the
// block a row is in or the other rows.
//
// What bounds it.  Decode reads each page once: 256 requests of 512 to 8192 tokens,
// 32 heads over 8 of 128, take 399 us, 5.8 TB/s, 0.85 of what a copy reaches.  A chunk
// per warp is one pass: scores to shared memory, the maxima, weights, P V; blocks of at
// most 8 rows have four CTAs per SM (128 registers), each warp with three pages in
// flight, which cover each other's latencies, and the issue slots are 49 % busy.  With
// the rows as M of the products, 12 of 16 were empty here: 424 us.  Four pages in flight
// and three CTAs, or two and five, are slower; pages loaded straight to registers take
// 467 to 528 us; resident CTAs that take blocks off a count gained 1.
// At head dimension 256 the registers allow two CTAs of such blocks: a window of 1024
// keys for 48 requests of 3 tokens, 8 heads over 4 (6 rows), 28 us, 3.8 TB/s, two rounds
// of latency.  Blocks of 9 to 16 rows take 91 KB of shared memory at 128 dims and 140 at
// 256, two CTAs per SM and one; a launch has one kind, by its largest block.
#include <math.h>

#include "attn_tile.cuh"
#include "kv8.cuh"
#include "vd_internal.h"

namespace vd {
namespace {

constexpr int kSplit8 = 512;   // keys of a split
constexpr int kChunk8 = 128;   // keys of a chunk
constexpr int kChunkPages = kChunk8 / 16;

// NB: the block's rows in groups of 8 (1 or 2).  Keys, and for P V the dims, are
// the M of the products and the rows their N, so that a block of few rows (4 per
// token at four heads per KV head) leaves little of them empty.
template <int HD, int NB>
struct Attn8Cfg {
  static constexpr int PART = Kv8Cfg<HD>::PART;
  static constexpr int SL = NB == 1 ? 3 : 4;        // copies in flight per warp
  static constexpr int OWN = 2 * 32 * HD;           // K and V of one bf16 page
  static constexpr int RING = SL * PART;            // per warp
  static_assert(RING >= 8 * NB * HD * 4, "the chunk's O, [row][HD], takes the place of the copies");
  // per warp: the scores, [page][lane][row group]: keys g, g + 8 of rows 2t, 2t + 1
  static constexpr int SC = (kChunkPages + 2) * 32 * NB * 16;
  static constexpr int smem(int own_slots) { return 1024 + own_slots * OWN + 4 * (RING + SC) + (4 * SL + 2) * 8 + 16; }
};

__device__ __forceinline__ uint32_t transpose8(uint32_t v) {  // an 8 x 8 fragment of fp16
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <int HD, int FMT, int NB>
__global__ void __launch_bounds__(128, HD <= 128 ? (NB == 1 ? 4 : 3) : 2)
    attn8_kernel(const __grid_constant__ CUtensorMap kvmap, Attn8Args a) {
  using C = Attn8Cfg<HD, NB>;
  constexpr int NR = 2 * NB, SL = C::SL, KK = HD / 16, UNITS = Kv8Cfg<HD>::UNITS;  // NR: rows per lane
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, t4 = lane & 3;
  uint8_t* own_s = smem;
  uint8_t* ring0 = smem + a.own_slots * C::OWN;
  uint8_t* ring = ring0 + warp * C::RING;
  uint8_t* score_s = ring0 + 4 * C::RING;
  float4* score = reinterpret_cast<float4*>(score_s + warp * C::SC) + lane * NB;  // page i at score[i * 32 * NB]
  uint64_t* bars = reinterpret_cast<uint64_t*>(score_s + 4 * C::SC);
  uint64_t* bar = bars + warp * SL;
  uint64_t* own_bar = bars + 4 * SL;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(own_bar + 2);
  __shared__ float2 fold_m[4][8 * NB];
  __shared__ float fold_l[kChunkParts][4][8 * NB];  // per chunk and row: its Kv8Max, its parts' l

  // Up to the wait for the previous kernel the CTA reads only the status word and
  // the plan (uploaded before the step's first kernel).
  __shared__ int skip;
  if (threadIdx.x == 0) {
    skip = a.status ? *reinterpret_cast<volatile int*>(a.status) : 0;
    for (int k = 0; k < 4 * SL + 2; ++k) mbar_init(&bars[k], 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  // The block: its request, rows and split come from the plan in one round trip
  // (a search over the requests took three), and with them a decode block's pages;
  // the KV heads of one split side by side, so that CTAs in flight together read
  // whole pages.
  const int kvh = blockIdx.x % a.Hkv;
  const int item = blockIdx.x / a.Hkv;
  const int4 d0 = a.items[2 * item], d1 = a.items[2 * item + 1];
  int pid = 0, opid = 0;  // lane i: the page a8 + i in 8 bits, ao + i in bf16
  if (a.split_pages && lane < kChunkPages) pid = a.split_pages[item * (kSplit8 / 16) + warp * kChunkPages + lane];
  const int b = d0.x, q0 = d0.y, qlen = d0.z, cached = d0.w, sidx = d1.x, r0 = d1.y, part0 = d1.w;
  const int G = a.Hq / a.Hkv;
  const int rows = qlen * G;
  const int r_end = min(rows, r0 + 16);
  const int p_min = cached + r0 / G, p_max = cached + (r_end - 1) / G;
  const int lo_min = a.window > 0 ? max(0, p_min - a.window + 1) : 0;
  // this warp's chunk: pages [a8, a8 + n8) in 8 bits, [ao, ao + no) in bf16
  const int pg0 = (sidx * kSplit8 + warp * kChunk8) >> 4;
  const int own_lo = p_min >> 4, own_hi = p_max >> 4;
  const int a8 = max(pg0, lo_min >> 4), n8 = max(0, min(pg0 + kChunkPages, own_hi) - a8);
  const int ao = max(pg0, own_lo), no = max(0, min(pg0 + kChunkPages - 1, own_hi) - ao + 1);
  if (a.split_pages) pid = __shfl_sync(0xffffffffu, pid, (lane + a8 - pg0) & 31);
  else if (lane < n8) pid = a.page_table[static_cast<size_t>(b) * a.pt_stride + a8 + lane];
  if (lane < no) opid = a.open_table[static_cast<size_t>(b) * a.open_stride + ao + lane - (cached >> 4)];
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  if (skip) return;
  if (max(sidx * kSplit8, lo_min) > min(sidx * kSplit8 + kSplit8 - 1, p_max)) return;  // no visible key of these rows

  // Copies of this warp: its K pages, then its V pages, copy j into slot j % SL,
  // issued by the lane that holds the page's id.  (Straight from memory into
  // registers, which the codes' order allows, with as many bytes in flight, the
  // kernel took 10 to 25 % longer: the loads of a whole page then have to be
  // waited for where its first word is used.)
  const uint8_t* page = a.codes + (static_cast<size_t>(pid) * a.Hkv + kvh) * (2 * C::PART);
  auto issue = [&](int j, bool v) {
    uint64_t* f = &bar[j % SL];
    mbar_arrive_expect_tx(f, C::PART);
    bulk_load(ring + (j % SL) * C::PART, page + (v ? C::PART : 0), C::PART, f);
  };
  if (lane < n8 && lane < SL) issue(lane, false);
  if (lane < n8 && n8 + lane < SL) issue(n8 + lane, true);
  int issued = min(SL, 2 * n8);
  if (lane < no) {
    const int o = ao + lane - own_lo, row = a.layer_row0 + ((opid * 2) * a.Hkv + kvh) * 16;
    mbar_arrive_expect_tx(&own_bar[o], C::OWN);
    tma_load_3d(own_s + o * C::OWN, &kvmap, &own_bar[o], 0, 0, row);
    tma_load_3d(own_s + o * C::OWN + C::OWN / 2, &kvmap, &own_bar[o], 0, 0, row + a.Hkv * 16);
  }
  float4 sc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (lane < n8) sc = __ldcg(a.scales + static_cast<size_t>(pid) * a.Hkv + kvh);

  // ---- the rows' queries as fp16 B fragments (lane: row g of each group), and
  // what this lane needs of the rows whose scores it gets, 2t and 2t + 1 of each
  uint32_t qf[KK][NB][2];
  float rowfac[NR];
  int pos[NR], lo[NR], own[NR];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int row = r0 + 8 * n + gq;
    const bool valid = row < rows;
    const __nv_bfloat16* qr = a.q + (static_cast<size_t>(q0 + row / G) * a.Hq + kvh * G + row % G) * HD + t4 * 2;
    uint32_t mx = 0u;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      qf[kk][n][0] = valid ? *reinterpret_cast<const uint32_t*>(qr + kk * 16) : 0u;
      qf[kk][n][1] = valid ? *reinterpret_cast<const uint32_t*>(qr + kk * 16 + 8) : 0u;
    }
#pragma unroll
    for (int kk = 0; kk < KK; ++kk)
      mx = __vmaxu2(mx, __vmaxu2(qf[kk][n][0] & 0x7fff7fffu, qf[kk][n][1] & 0x7fff7fffu));
    mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int e = kv8_exp(kv8_max_halves(mx));
    const float up = kv8_up(e), fac = e == 255 ? kv8_nan() : __fmul_rn(a.scale_log2, kv8_down(e));
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      qf[kk][n][0] = kv8_to_f16(qf[kk][n][0], up);
      qf[kk][n][1] = kv8_to_f16(qf[kk][n][1], up);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = 2 * n + k, rr = r0 + 8 * n + 2 * t4 + k;
      rowfac[r] = __shfl_sync(0xffffffffu, fac, (2 * t4 + k) * 4);
      pos[r] = rr < rows ? cached + rr / G : -1;
      own[r] = pos[r] >> 4;  // -1 for a row that is none
      lo[r] = rr < rows ? (a.window > 0 ? max(0, pos[r] - a.window + 1) : 0) : 1;
    }
  }

  bool ok = true;
  auto wait = [&](uint64_t* f, uint32_t parity) {
    ok = ok && __all_sync(0xffffffffu, mbar_wait(f, parity, abort_flag, a.status));
    return ok;
  };
  int used = 0;  // copies waited for
  // The slot of copy j is free: copy j + SL goes there.
  auto refill = [&](int j) {
    const int k = j + SL;
    if (k < 2 * n8) {
      if (lane == (k < n8 ? k : k - n8)) issue(k, k >= n8);
      issued = k + 1;
    }
  };
  // Pages whose every key every row of the block sees (rows that are none aside)
  // take no masking: [full_lo, own_lo).
  const int full_lo = a.window > 0 ? (max(0, p_max - a.window + 1) + 15) >> 4 : 0;
  auto full = [&](int pg) { return pg >= full_lo && pg < own_lo; };

  // ---- scores of the 8-bit pages, two at a time; the odd last one is taken
  // twice.  Element e of a score fragment: key g + 8 (e / 2), row 2t + e % 2.
  Kv8Max mx[NR];
#pragma unroll 1
  for (int i = 0; i < n8; i += 2) {
    const int i1 = min(i + 1, n8 - 1);
    if (!wait(&bar[i % SL], (i / SL) & 1) || !wait(&bar[i1 % SL], (i1 / SL) & 1)) break;
    used = i1 + 1;
    const uint4* kp0 = reinterpret_cast<const uint4*>(ring + (i % SL) * C::PART) + lane;
    const uint4* kp1 = reinterpret_cast<const uint4*>(ring + (i1 % SL) * C::PART) + lane;
    float acc[2][NB][4];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int n = 0; n < NB; ++n) acc[x][n][0] = acc[x][n][1] = acc[x][n][2] = acc[x][n][3] = 0.f;
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const uint4 w[2] = {kp0[u * 32], kp1[u * 32]};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t f[4];
        kv8_expand<FMT>(w[x].x, f[0], f[2]);
        kv8_expand<FMT>(w[x].y, f[1], f[3]);
#pragma unroll
        for (int n = 0; n < NB; ++n) mma_f16_16816(acc[x][n], f, qf[2 * u][n][0], qf[2 * u][n][1]);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t f[4];
        kv8_expand<FMT>(w[x].z, f[0], f[2]);
        kv8_expand<FMT>(w[x].w, f[1], f[3]);
#pragma unroll
        for (int n = 0; n < NB; ++n) mma_f16_16816(acc[x][n], f, qf[2 * u + 1][n][0], qf[2 * u + 1][n][1]);
      }
    }
    __syncwarp();
    refill(i);
    if (i1 > i) refill(i1);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int ii = x ? i1 : i, pgi = a8 + ii;
      const float ks = __shfl_sync(0xffffffffu, sc.x, ii), lv = __shfl_sync(0xffffffffu, sc.z, ii);
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __fmul_rn(acc[x][n][e], __fmul_rn(ks, rowfac[2 * n + (e & 1)]));
        if (!full(pgi)) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 2 * n + (e & 1), key = pgi * 16 + gq + 8 * (e >> 1);
            if (!(key >= lo[r] && pgi < own[r])) v[e] = -INFINITY;
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float s1 = fmaxf(v[k], v[2 + k]);
          kv8_take(mx[2 * n + k], s1, __fadd_rn(s1, lv));
        }
        score[ii * 32 * NB + n] = make_float4(v[0], v[1], v[2], v[3]);
      }
    }
  }
  // ---- scores of the own pages
  int ve[2][4];     // [own page][key]: the exponents of V tokens 2t, 2t + 1, 2t + 8, 2t + 9
  float vlv[2][2];  // [own page]: log2 of the V scales of tokens g, g + 8
  const int mi = lane >> 3, r8 = lane & 7;
#pragma unroll 1
  for (int o = 0; o < no; ++o) {
    const int oi = ao + o - own_lo;
    if (!wait(&own_bar[oi], 0)) break;
    const uint32_t kb = smem_u32(own_s + oi * C::OWN), vb = kb + C::OWN / 2;
    // largest magnitudes: of K tokens g and g + 8, then of V tokens 8 j + 2 t + {0, 1}
    uint32_t km[2] = {0u, 0u}, vm[2] = {0u, 0u};
#pragma unroll 4
    for (int kk = 0; kk < KK; ++kk) {
      uint32_t w[4];
      ldmatrix_x4(w, kb + kv_off<HD>((mi & 1) * 8 + r8, kk * 2 + (mi >> 1)));
      km[0] = __vmaxu2(km[0], __vmaxu2(w[0] & 0x7fff7fffu, w[2] & 0x7fff7fffu));
      km[1] = __vmaxu2(km[1], __vmaxu2(w[1] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
      ldmatrix_x4_trans(w, vb + kv_off<HD>((mi & 1) * 8 + r8, kk * 2 + (mi >> 1)));
      vm[0] = __vmaxu2(vm[0], __vmaxu2(w[0] & 0x7fff7fffu, w[2] & 0x7fff7fffu));
      vm[1] = __vmaxu2(vm[1], __vmaxu2(w[1] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
    }
    int vx[4];
    float kup[2], kd[2], lv[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      km[j] = __vmaxu2(km[j], __shfl_xor_sync(0xffffffffu, km[j], 1));
      km[j] = __vmaxu2(km[j], __shfl_xor_sync(0xffffffffu, km[j], 2));
      const int ke = kv8_exp(kv8_max_halves(km[j]));
      kup[j] = kv8_up(ke);
      kd[j] = ke == 255 ? kv8_nan() : kv8_down(ke);
#pragma unroll
      for (int x = 4; x < 32; x *= 2) vm[j] = __vmaxu2(vm[j], __shfl_xor_sync(0xffffffffu, vm[j], x));
      vx[2 * j] = kv8_exp(vm[j] & 0xffffu);
      vx[2 * j + 1] = kv8_exp(vm[j] >> 16);
      const int e0 = __shfl_sync(0xffffffffu, vx[2 * j], gq >> 1), e1 = __shfl_sync(0xffffffffu, vx[2 * j + 1], gq >> 1);
      const int e = gq & 1 ? e1 : e0;  // of token g + 8 j
      lv[j] = e == 255 ? kv8_nan() : kv8_log2_down(e);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (o == 0) ve[0][x] = vx[x];
      else ve[1][x] = vx[x];
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (o == 0) vlv[0][x] = lv[x];
      else vlv[1][x] = lv[x];
    }
    float acc[NB][4];
#pragma unroll
    for (int n = 0; n < NB; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      uint32_t w[4];
      ldmatrix_x4(w, kb + kv_off<HD>((mi & 1) * 8 + r8, kk * 2 + (mi >> 1)));
      const uint32_t f[4] = {kv8_to_f16(w[0], kup[0]), kv8_to_f16(w[1], kup[1]), kv8_to_f16(w[2], kup[0]), kv8_to_f16(w[3], kup[1])};
#pragma unroll
      for (int n = 0; n < NB; ++n) mma_f16_16816(acc[n], f, qf[kk][n][0], qf[kk][n][1]);
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 2 * n + (e & 1), key = (ao + o) * 16 + gq + 8 * (e >> 1);
        const bool vis = key >= lo[r] && key <= pos[r] && ao + o == own[r];
        v[e] = vis ? __fmul_rn(acc[n][e], __fmul_rn(kd[e >> 1], rowfac[r])) : -INFINITY;
        kv8_take(mx[r], v[e], __fadd_rn(v[e], lv[e >> 1]));
      }
      score[(kChunkPages + o) * 32 * NB + n] = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
  // ---- the running maxima of the split at this chunk
#pragma unroll
  for (int r = 0; r < NR; ++r) {
#pragma unroll
    for (int x = 4; x < 32; x *= 2)
      kv8_take(mx[r], __shfl_xor_sync(0xffffffffu, mx[r].s, x), __shfl_xor_sync(0xffffffffu, mx[r].t, x));
    if (gq == 0) fold_m[warp][8 * (r >> 1) + 2 * t4 + (r & 1)] = make_float2(mx[r].s, mx[r].t);
  }
  __syncthreads();
  Kv8Base base[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    for (int w = 0; w < warp; ++w) {
      const float2 m = fold_m[w][8 * (r >> 1) + 2 * t4 + (r & 1)];
      kv8_take(mx[r], m.x, m.y);
    }
    base[r] = Kv8Base(mx[r], kv8_exponent(mx[r]));
  }

  // ---- weights, their sums and P V
  float l[NR][kChunkParts], o_acc[HD / 16][NB][4];  // element e of O: dim 16 x + g + 8 (e / 2), row 2t + e % 2
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int h = 0; h < kChunkParts; ++h) l[r][h] = 0.f;
#pragma unroll
  for (int x = 0; x < HD / 16; ++x)
#pragma unroll
    for (int n = 0; n < NB; ++n) o_acc[x][n][0] = o_acc[x][n][1] = o_acc[x][n][2] = o_acc[x][n][3] = 0.f;
  // Weights of page `pg`, at place i of the scores, as B fragments, and their share of l;
  // of(r, j): row r's Kv8Weight of token g + 8 j.
  auto weights = [&](int i, int pg, auto of, uint32_t (&pb)[NB][2]) {
    const int part = (pg - pg0) / (kChunkPages / kChunkParts);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const float4 v = score[i * 32 * NB + n];
      const float s4[4] = {v.x, v.y, v.z, v.w};
      float p[4], back[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const Kv8Weight w = of(2 * n + (e & 1), e >> 1);
        p[e] = ex2(__fsub_rn(s4[e], w.base));
        back[e] = w.back;
      }
      pb[n][0] = transpose8(pack_f16x2(p[0], p[1]));
      pb[n][1] = transpose8(pack_f16x2(p[2], p[3]));
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int h = 0; h < kChunkParts; ++h)
          if (h == part) l[2 * n + k][h] = __fmaf_rn(p[2 + k], back[2 + k], __fmaf_rn(p[k], back[k], l[2 * n + k][h]));
    }
  };
#pragma unroll 1
  for (int i = 0; i < n8; ++i) {
    const int cp = n8 + i;  // the copy of page i's V
    uint32_t pb[NB][2];
    const float lv = __shfl_sync(0xffffffffu, sc.z, i);
    const int pg = a8 + i;
    const bool all = full(pg);
    Kv8Weight w[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r)  // (a page that the row does not see stays out, whatever its scale)
      w[r] = all || (pg < own[r] && pg * 16 + 15 >= lo[r]) ? base[r](lv) : kv8_no_weight();
    weights(i, pg, [&](int r, int) { return w[r]; }, pb);
    if (!wait(&bar[cp % SL], (cp / SL) & 1)) break;
    used = cp + 1;
    const uint4* vp = reinterpret_cast<const uint4*>(ring + (cp % SL) * C::PART) + lane;
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const uint4 w = vp[u * 32];
      uint32_t f[4];
      kv8_expand<FMT>(w.x, f[0], f[2]);
      kv8_expand<FMT>(w.y, f[1], f[3]);
#pragma unroll
      for (int n = 0; n < NB; ++n) mma_f16_16816(o_acc[2 * u][n], f, pb[n][0], pb[n][1]);
      kv8_expand<FMT>(w.z, f[0], f[2]);
      kv8_expand<FMT>(w.w, f[1], f[3]);
#pragma unroll
      for (int n = 0; n < NB; ++n) mma_f16_16816(o_acc[2 * u + 1][n], f, pb[n][0], pb[n][1]);
    }
    __syncwarp();
    refill(cp);
  }
  if (ok) {
#pragma unroll 1
    for (int o = 0; o < no; ++o) {
      const uint32_t vb = smem_u32(own_s + (ao + o - own_lo) * C::OWN + C::OWN / 2);
      float up[4];                  // of keys 2t, 2t + 1, 2t + 8, 2t + 9
      uint32_t keep[2] = {0u, 0u};  // fp16 pairs: a token that is not finite counts as 0 here (its weight is NaN, or 0)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int e = o == 0 ? ve[0][x] : ve[1][x];
        up[x] = kv8_up(e);
        if (e != 255) keep[x >> 1] |= 0xffffu << (16 * (x & 1));
      }
      uint32_t pb[NB][2];
      const int pg = ao + o;
      const float lv[2] = {o == 0 ? vlv[0][0] : vlv[1][0], o == 0 ? vlv[0][1] : vlv[1][1]};
      weights(kChunkPages + o, pg, [&](int r, int j) {  // (a token that the row does not see stays out)
        const int key = pg * 16 + gq + 8 * j;
        return pg == own[r] && key >= lo[r] && key <= pos[r] ? base[r](lv[j]) : kv8_no_weight();
      }, pb);
#pragma unroll
      for (int x = 0; x < HD / 16; ++x) {
        uint32_t w[4];
        ldmatrix_x4_trans(w, vb + kv_off<HD>((mi & 1) * 8 + r8, x * 2 + (mi >> 1)));
        uint32_t f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)  // (dims 8 (k / 2) on, keys 8 (k % 2) on) -> fragment register k / 2 + 2 (k % 2)
          f[(k >> 1) + 2 * (k & 1)] =
              pack_f16x2(__fmul_rn(bf16_lo(w[k]), up[2 * (k & 1)]), __fmul_rn(bf16_hi(w[k]), up[2 * (k & 1) + 1])) & keep[k & 1];
#pragma unroll
        for (int n = 0; n < NB; ++n) mma_f16_16816(o_acc[x][n], f, pb[n][0], pb[n][1]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int h = 0; h < kChunkParts; ++h) {
      float x = l[r][h];
#pragma unroll
      for (int k = 4; k < 32; k *= 2) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, k));
      if (gq == 0) fold_l[h][warp][8 * (r >> 1) + 2 * t4 + (r & 1)] = x;
    }
  if (!ok) {  // gave up: every copy lands before the warp leaves
    for (int j = used; j < issued; ++j) drain_wait(&bar[j % SL], (j / SL) & 1);
    for (int o = 0; o < no; ++o) drain_wait(&own_bar[ao + o - own_lo], 0);
  }

  // ---- the chunks of the split, left to right.  Each warp's O takes the place of
  // its copies; 8-float groups of a row are XORed with the row's pair, so that the
  // stores of a warp meet no bank twice.
  __syncwarp();
  float* fo = reinterpret_cast<float*>(ring);  // [row][HD]
#pragma unroll
  for (int x = 0; x < HD / 16; ++x)
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        fo[(8 * n + 2 * t4 + (e & 1)) * HD + ((16 * x + 8 * (e >> 1)) ^ (8 * t4)) + gq] = o_acc[x][n][e];
  __syncthreads();
  if (*abort_flag) return;
  constexpr int TPR = 128 / (8 * NB), PER = HD / TPR;  // threads and dims per row
  const int frow = threadIdx.x / TPR, fd = threadIdx.x % TPR;
  const int row = r0 + frow;
  if (row >= rows) return;
  Kv8Max M;
  float M_ex = 0.f, L[kChunkParts] = {}, O[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) O[i] = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float* src = reinterpret_cast<const float*>(ring0 + w * C::RING) + frow * HD;
    float al, ao;
    const float s0 = M.s;
    kv8_take(M, fold_m[w][frow].x, fold_m[w][frow].y);
    kv8_factors(M, s0, M_ex, al, ao);
#pragma unroll
    for (int h = 0; h < kChunkParts; ++h) L[h] = __fmaf_rn(L[h], al, fold_l[h][w][frow]);
#pragma unroll
    for (int i = 0; i < PER / 4; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(src + (((i * TPR + fd) * 4) ^ (8 * ((frow >> 1) & 3))));
      O[4 * i] = __fmaf_rn(O[4 * i], ao, v.x);
      O[4 * i + 1] = __fmaf_rn(O[4 * i + 1], ao, v.y);
      O[4 * i + 2] = __fmaf_rn(O[4 * i + 2], ao, v.z);
      O[4 * i + 3] = __fmaf_rn(O[4 * i + 3], ao, v.w);
    }
  }
  // a row that sees no key of the split has no partial
  const int p = cached + row / G, flo = a.window > 0 ? max(0, p - a.window + 1) : 0;
  if (max(flo, sidx * kSplit8) > min(p, sidx * kSplit8 + kSplit8 - 1)) return;
  const size_t at = (static_cast<size_t>(part0 + row / G) * a.Hq + kvh * G + row % G) * a.max_splits + sidx;
  if (fd == 0) {
    a.part_ml[at * 2] = M.s;
    a.part_ml[at * 2 + 1] = __fmul_rn(kv8_sum_parts(L), kPart);
  }
  const float unit = ex2(__fadd_rn(M_ex, kPartLog2));
#pragma unroll
  for (int i = 0; i < PER / 4; ++i)
    *reinterpret_cast<float4*>(a.part_o + at * HD + (i * TPR + fd) * 4) =
        make_float4(kv8_part(O[4 * i], unit), kv8_part(O[4 * i + 1], unit), kv8_part(O[4 * i + 2], unit),
                    kv8_part(O[4 * i + 3], unit));
}

template <int HD, int FMT, int NB>
int launch_attn8_t(const CUtensorMap& kvmap, const Attn8Args& a, int n_blocks, cudaStream_t s) {
  using C = Attn8Cfg<HD, NB>;
  static_assert(C::smem(2) + 1024 <= 227 * 1024, "shared memory");
  VD_CUDA_TRY(cudaFuncSetAttribute(attn8_kernel<HD, FMT, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(2)));
  VD_CUDA_TRY(launch_k(attn8_kernel<HD, FMT, NB>, dim3(static_cast<unsigned>(n_blocks) * a.Hkv), dim3(128), C::smem(a.own_slots), s, kvmap, a));
  return VD_OK;
}

}  // namespace

static_assert(kAttn8Split == kSplit8, "split of the plan's items");

int launch_attention8(const CUtensorMap& kvmap, const Attn8Args& a, int hd, int format, bool lower8, int n_blocks,
                      cudaStream_t s) {
  if (n_blocks <= 0) return VD_OK;
#define VD_ATTN8(HD_)                                                                                             \
  if (hd == HD_) {                                                                                                \
    if (format == VD_KV8_INT8)                                                                                    \
      return lower8 ? launch_attn8_t<HD_, kKv8Int8, 1>(kvmap, a, n_blocks, s)                                   \
                    : launch_attn8_t<HD_, kKv8Int8, 2>(kvmap, a, n_blocks, s);                                 \
    return lower8 ? launch_attn8_t<HD_, kKv8E4m3, 1>(kvmap, a, n_blocks, s)                                     \
                  : launch_attn8_t<HD_, kKv8E4m3, 2>(kvmap, a, n_blocks, s);                                   \
  }
  VD_ATTN8(64)
  VD_ATTN8(128)
  VD_ATTN8(256)
#undef VD_ATTN8
  return fail(VD_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
}

}  // namespace vd
