// A whole mixture-of-experts layer for a few tokens (gfx950).
//
//   gate, up = blockwise(A[t], W_gate_up[e])         exact int32 per 128 of K
//   hq, hs   = group quantiser of silu(gate) * up    fp32, groups of 128
//   Y[t]     = sum_j w[t][j] blockwise(hq, W_down[e])  over the token's slots
//
// The block-wise scheme is section 2.3 of "DeepSeek R1 INT8 quantisation in
// SGLang" (Meituan) applied per expert; that DeepSeek's feed-forward layers
// are mixtures of experts is stated on "FP8 vs INT8 quantisation for
// DeepSeek", section 1.2.
//
// With at most 64 tokens the experts' weights are nearly all of the traffic
// (3 I K bytes for each expert that a token chose), so two kernels stream
// them once, straight from global memory into MFMA operand registers:
// k_moe_gate_up and k_moe_down.  Between them h is quantised, by the down
// kernel itself where the pairs are few, else by k_moe_quant; where the output
// has few columns, k_moe_combine sums what several down workgroups share.
// 64 tokens, K = 7168, I = 2048, 64 experts, 8 of them per token (2.8 GB of
// weights, each byte fetched once by the counters): 313 + 5 + 162 us, 6.0 and
// 5.8 TB/s; one token (352 MB): 43 + 26 us.
//
// A "pair" is one slot of one token (t, j), p = t topk + j; the pairs of one
// expert are the rows of its products, in the order of p, and the rows of all
// experts in the order of the expert index are the rows of hq.  A pair whose
// id is outside 0 .. E - 1 has no row.  Which variant of each kernel a call
// takes stands in moe_plan.h.
#include "common.h"
#include "launch.h"
#include "moe_plan.h"

namespace w8 {
namespace {

typedef __amdgpu_buffer_rsrc_t rsrc_t;

// Added to the offset of a load that must read zero: beyond the range of
// every descriptor here (at most 1024 rows x 2^15 bytes), twice it still
// inside 32 bits.
constexpr uint32_t kOob = 0x40000000u;

// Base and size are uniform; readfirstlane keeps the descriptor in scalar
// registers.  Loads past `bytes` return zero and move no data.
__device__ __forceinline__ rsrc_t rsrc(const void* base, int64_t bytes) {
  const uint64_t a = (uint64_t)base;
  const uint64_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  const uint64_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
  const int n = __builtin_amdgcn_readfirstlane((int)bytes);
  return __builtin_amdgcn_make_buffer_rsrc((void*)(lo | (hi << 32)), 0, n, 0x00020000);
}
__device__ __forceinline__ v4i bl16(rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}
__device__ __forceinline__ float blf(rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0));
}

__device__ __forceinline__ v4f block_fma(v4f acc, v4i w0, v4i w1, v4i a0, v4i a1, float s) {
  v4i p = __builtin_amdgcn_mfma_i32_16x16x64_i8(w0, a0, (v4i){0, 0, 0, 0}, 0, 0, 0);
  p = __builtin_amdgcn_mfma_i32_16x16x64_i8(w1, a1, p, 0, 0, 0);
#pragma unroll
  for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(s, (float)p[r], acc[r]);
  return acc;
}

// ------------------------------------------------------------- gate and up
// Wave fragments (v_mfma_i32_16x16x64_i8, weights as operand A): lane l holds
// weight row l & 15 and activation row l & 15, bytes 16 (l >> 4) .. +15 of
// each 64-wide half of the K block; the result lane holds columns
// 4 (l >> 4) .. +3 of activation row l & 15.
//
// Sums over the K blocks par, par + WK, ... of rows r0 .. r0 + 16 MF - 1 of
// expert e against its gate columns c0 .. c0 + 16 FC - 1 (acc[f], f < FC) and
// the up columns of the same index (acc[FC + f]).  PF blocks of loads stay in
// flight in a register ring.  A CU's loads are limited by their number as
// much as by their bytes, so the ring holds codes only: the scales of the
// rows (sx, rows KB | 1 floats apart) and of the columns (sw, gate then up)
// lie in LDS.
template <int MF, int FC, int PF, int WK, class F>
__device__ __forceinline__ void gate_up_sums(const MoeArgs& a, int e, int c0, int par, int r0, int n,
                                             const uint16_t* tok, const float* sx, const float* sw, F stage,
                                             v4f (&acc)[2 * FC][MF]) {
  const int lane = threadIdx.x & 63;
  const int q = lane >> 4;
  const int K = a.K, KB = K >> 7;
  const int64_t wrow = (int64_t)e * 2 * a.I + c0;
  const rsrc_t rg = rsrc(a.w13 + wrow * K, (int64_t)16 * FC * K);
  const rsrc_t ru = rsrc(a.w13 + (wrow + a.I) * K, (int64_t)16 * FC * K);
  const rsrc_t ra = rsrc(a.A, (int64_t)a.T * K);
  const uint32_t woff = (uint32_t)((lane & 15) * K + q * 16);
  uint32_t aoff[MF];
#pragma unroll
  for (int j = 0; j < MF; ++j) {
    const int r = r0 + 16 * j + (lane & 15);
    aoff[j] = r < n ? (uint32_t)tok[r < n ? r : 0] * (uint32_t)K + q * 16 : kOob;
  }
#pragma unroll
  for (int f = 0; f < 2 * FC; ++f)
#pragma unroll
    for (int j = 0; j < MF; ++j) acc[f][j] = (v4f){0.f, 0.f, 0.f, 0.f};

  v4i wv[PF][2 * FC][2], av[PF][MF][2];
  auto load = [&](int P, int kb) {
    const uint32_t ko = kb < KB ? (uint32_t)kb * 128u : kOob;
#pragma unroll
    for (int f = 0; f < FC; ++f) {
      const uint32_t at = woff + (uint32_t)(16 * f * K) + ko;
      wv[P][f][0] = bl16(rg, at);
      wv[P][f][1] = bl16(rg, at + 64);
      wv[P][FC + f][0] = bl16(ru, at);
      wv[P][FC + f][1] = bl16(ru, at + 64);
    }
#pragma unroll
    for (int j = 0; j < MF; ++j) {
      av[P][j][0] = bl16(ra, aoff[j] + ko);
      av[P][j][1] = bl16(ra, aoff[j] + ko + 64);
    }
  };
#pragma unroll
  for (int p = 0; p < PF; ++p) {
    load(p, par + WK * p);
    __builtin_amdgcn_sched_barrier(0);
  }
  stage();
  // a block past the last multiplies zero codes, with the last one's scales
  for (int kb = par; kb < KB; kb += WK * PF) {
#pragma unroll
    for (int p = 0; p < PF; ++p) {
      const int kc = kb + WK * p < KB ? kb + WK * p : KB - 1;
      const float sg = sw[kc], su = sw[KB + kc];
#pragma unroll
      for (int j = 0; j < MF; ++j) {
        const float x = sx[(16 * j + (lane & 15)) * (KB | 1) + kc];
#pragma unroll
        for (int f = 0; f < 2 * FC; ++f)
          acc[f][j] = block_fma(acc[f][j], wv[p][f][0], wv[p][f][1], av[p][j][0], av[p][j][1],
                                __fmul_rn(x, f < FC ? sg : su));
      }
      load(p, kb + WK * (p + PF));
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

__device__ __forceinline__ v4f silu_mul(v4f g, v4f u) {
  v4f h;
#pragma unroll
  for (int r = 0; r < 4; ++r) h[r] = g[r] / (1.0f + expf(-g[r])) * u[r];
  return h;
}

// The group quantiser of 16 of a group's values per lane, 8 lanes per group.
// h is quantised from fp32 (a 16-bit h would be read by nobody).
__device__ __forceinline__ uint4 quant16(const float4* raw, float* scale) {
  float v[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[4 * i] = raw[i].x;
    v[4 * i + 1] = raw[i].y;
    v[4 * i + 2] = raw[i].z;
    v[4 * i + 3] = raw[i].w;
  }
  const QScale sc = make_scale(max8(amax_n(v, 16)));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = quant_one(v[i], sc);
  *scale = sc.s;
  return make_uint4(pack4(v[0], v[1], v[2], v[3]), pack4(v[4], v[5], v[6], v[7]), pack4(v[8], v[9], v[10], v[11]),
                    pack4(v[12], v[13], v[14], v[15]));
}

// ---------------------------------------------------- who has which expert
constexpr int kGuThreads = 64 * kGuWaves;
constexpr int kPerThread = kMaxPairs / kGuThreads;

struct Chosen {
  int e, n, base;   // an expert, its rows, the rows of lower experts; e < 0: none
};

// The k-th of the chosen experts, counted in the order of their first pairs,
// from the ids alone; tok[r] becomes the token of its row r.  owner holds E
// ints of LDS: the least pair of each chosen expert.  With `table` the layer's
// tables for the later kernels are written too: each pair's row (pos, -1 if
// it has none), and this expert's index, rows (count, 0 if there is no k-th
// expert) and first row.  Every thread of the workgroup calls it.
__device__ __forceinline__ Chosen choose(const MoeArgs& a, int k, bool table, int* owner, uint16_t* tok) {
  __shared__ int cnt[3][kPerThread * kGuWaves];
  __shared__ int sel;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int P = a.T * a.topk;
  const int parts = (P + kGuThreads - 1) / kGuThreads;   // of 256 pairs
  int id[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int p = i * kGuThreads + threadIdx.x;
    id[i] = p < P ? a.ids[p] : -1;
    if (id[i] < 0 || id[i] >= a.E) id[i] = -1;
    if (id[i] >= 0) owner[id[i]] = kMaxPairs;
  }
  if (threadIdx.x == 0) sel = -1;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPerThread; ++i)
    if (id[i] >= 0) atomicMin(&owner[id[i]], i * kGuThreads + (int)threadIdx.x);
  __syncthreads();
  uint64_t firsts[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    if (i >= parts) break;
    firsts[i] = __ballot(id[i] >= 0 && owner[id[i] < 0 ? 0 : id[i]] == i * kGuThreads + (int)threadIdx.x);
    if (lane == 0) cnt[0][i * kGuWaves + wave] = __popcll(firsts[i]);
  }
  __syncthreads();
  int active = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    if (i >= parts) break;
#pragma unroll
    for (int w = 0; w < kGuWaves; ++w) {
      const int c = cnt[0][i * kGuWaves + w];
      if (w == wave && (firsts[i] >> lane & 1) && active + __popcll(firsts[i] & ((1ull << lane) - 1)) == k)
        sel = id[i];
      active += c;
    }
  }
  __syncthreads();
  Chosen c;
  c.e = __builtin_amdgcn_readfirstlane(sel);
  c.n = 0;
  c.base = 0;
  if (table && k == 0) {
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int p = i * kGuThreads + threadIdx.x;
      if (p < P && id[i] < 0) a.pos[p] = -1;
    }
  }
  if (c.e < 0) {
    if (table && threadIdx.x == 0) a.count[k] = 0;
    return c;
  }
  uint64_t mine[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    if (i >= parts) break;
    mine[i] = __ballot(id[i] == c.e);
    const uint64_t less = __ballot(id[i] >= 0 && id[i] < c.e);
    if (lane == 0) {
      cnt[1][i * kGuWaves + wave] = __popcll(mine[i]);
      cnt[2][i * kGuWaves + wave] = __popcll(less);
    }
  }
  __syncthreads();
  int row[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    if (i >= parts) break;
#pragma unroll
    for (int w = 0; w < kGuWaves; ++w) {
      if (w == wave) row[i] = c.n + __popcll(mine[i] & ((1ull << lane) - 1));
      c.n += cnt[1][i * kGuWaves + w];
      c.base += cnt[2][i * kGuWaves + w];
    }
  }
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int p = i * kGuThreads + threadIdx.x;
    if (i < parts && id[i] == c.e) {
      tok[row[i]] = (uint16_t)(p / a.topk);
      if (table) a.pos[p] = c.base + row[i];
    }
  }
  if (table && threadIdx.x == 0) {
    a.expert[k] = c.e;
    a.count[k] = c.n;
    a.start[k] = c.base;
  }
  __syncthreads();
  c.n = __builtin_amdgcn_readfirstlane(c.n);
  c.base = __builtin_amdgcn_readfirstlane(c.base);
  return c;
}

// Grid (I / (16 FC 4 / WK), min(pairs, E)).  The four waves of a workgroup
// split 16 FC 4 / WK columns of h of one expert, WK of them sharing 16 FC
// columns and splitting the K blocks.  A workgroup this small keeps the load
// of the CUs even: each CU streams at a rate of its own (its outstanding
// loads over the memory's latency, some 23 GB/s when all are at it), so the
// kernel takes as long as the CU with the most to load (128-column
// workgroups, one pass more than their number filled, 138 us where these take
// 102: 8 tokens, K = 4096, I = 1536).  The 128 columns of a quantisation group
// may lie in several workgroups; h leaves in fp32 and is quantised by its
// readers.
template <int MF, int FC, int PF, int WK>
__device__ __forceinline__ void gate_up_rows(const MoeArgs& a, const Chosen& c, int r0, const uint16_t* tok,
                                             float* lds) {
  constexpr int TILES = kGuWaves / WK;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave % WK, tile = wave / WK;
  const int c0 = (blockIdx.x * TILES + tile) * 16 * FC;
  const int KB = a.K >> 7;
  float* sw = lds;
  float* sx = sw + 2 * KB;
  // the scales of the first 64 K blocks are on their way before the ring (a
  // wait for a later load would wait for all of the ring's): wave 0 the gate
  // columns', wave 1 the up columns', wave w the rows w, w + 4, ...; rows past
  // the last read zeros
  const rsrc_t rs = rsrc(a.s13 + (int64_t)c.e * 2 * (a.I >> 7) * KB, (int64_t)2 * (a.I >> 7) * KB * 4);
  const rsrc_t rsa = rsrc(a.sa, (int64_t)a.T * KB * 4);
  const uint32_t swoff = wave < 2 ? (uint32_t)((wave * (a.I >> 7) + (c0 >> 7)) * KB * 4) : kOob;
  uint32_t sxoff[4 * MF];
#pragma unroll
  for (int j = 0; j < 4 * MF; ++j) {
    const int r = r0 + wave + kGuWaves * j;
    sxoff[j] = r < c.n ? (uint32_t)tok[r < c.n ? r : 0] * (uint32_t)KB * 4u : kOob;
  }
  float psw, psx[4 * MF];
  auto fetch = [&](int i) {
    const uint32_t o = i < KB ? (uint32_t)i * 4u : kOob;
    psw = blf(rs, swoff + o);
#pragma unroll
    for (int j = 0; j < 4 * MF; ++j) psx[j] = blf(rsa, sxoff[j] + o);
  };
  fetch(lane);
  auto stage = [&] {
    for (int i = lane;; i += 64) {
      if (i < KB) {
        if (wave < 2) sw[wave * KB + i] = psw;
#pragma unroll
        for (int j = 0; j < 4 * MF; ++j) sx[(wave + kGuWaves * j) * (KB | 1) + i] = psx[j];
      }
      if (i - lane + 64 >= KB) break;
      fetch(i + 64);
    }
    __syncthreads();
  };
  v4f acc[2 * FC][MF];
  gate_up_sums<MF, FC, PF, WK>(a, c.e, c0, part, r0, c.n, tok, sx, sw, stage, acc);
  __syncthreads();   // the scales' place is free
  v4f* red = reinterpret_cast<v4f*>(lds) + tile * (WK - 1) * 2 * FC * MF * 64;
  if (part > 0) {
#pragma unroll
    for (int f = 0; f < 2 * FC; ++f)
#pragma unroll
      for (int j = 0; j < MF; ++j) red[(((part - 1) * 2 * FC + f) * MF + j) * 64 + lane] = acc[f][j];
  }
  __syncthreads();
  if (part == 0) {
#pragma unroll
    for (int w = 0; w < WK - 1; ++w)
#pragma unroll
      for (int f = 0; f < 2 * FC; ++f)
#pragma unroll
        for (int j = 0; j < MF; ++j) acc[f][j] += red[((w * 2 * FC + f) * MF + j) * 64 + lane];
#pragma unroll
    for (int j = 0; j < MF; ++j) {
      const int r = r0 + 16 * j + (lane & 15);
#pragma unroll
      for (int f = 0; f < FC; ++f)
        if (r < c.n)
          *reinterpret_cast<v4f*>(a.h32 + (int64_t)(c.base + r) * a.I + c0 + 16 * f + 4 * (lane >> 4)) =
              silu_mul(acc[f][j], acc[FC + f][j]);
    }
  }
  if (r0 + 16 * MF < c.n) __syncthreads();
}

// MFBIG: fragments of rows at a time for an expert of more than 16 rows.
template <int MFBIG, int FC, int WK>
__global__ __launch_bounds__(kGuThreads, MFBIG == 4 ? 2 : 4) void k_moe_gate_up(MoeArgs a) {
  __shared__ uint16_t tok[kMaxPairs];
  extern __shared__ __align__(16) float lds[];   // E ints, then the scales, then the waves' sums
  const Chosen c = choose(a, blockIdx.y, blockIdx.x == 0, reinterpret_cast<int*>(lds), tok);
  if (c.e < 0) return;
  if (c.n <= 16) {
    gate_up_rows<1, FC, FC == 1 ? 4 : 2, WK>(a, c, 0, tok, lds);
  } else {
    for (int r0 = 0; r0 < c.n; r0 += 16 * MFBIG) gate_up_rows<MFBIG, FC, 1, WK>(a, c, r0, tok, lds);
  }
}

// The codes and scales of h, a group per 8 lanes; rows behind the last pair's
// hold whatever the workspace held and nobody reads theirs.
__global__ __launch_bounds__(256) void k_moe_quant(MoeArgs a, int P, int IB) {
  const int groups = P * IB;
  const int g = blockIdx.x * 32 + (threadIdx.x >> 3), l8 = threadIdx.x & 7;
  const float4* at = reinterpret_cast<const float4*>(a.h32 + (int64_t)(g < groups ? g : groups - 1) * 128) + l8 * 4;
  const float4 raw[4] = {at[0], at[1], at[2], at[3]};
  float s;
  const uint4 o = quant16(raw, &s);
  if (g < groups) {
    reinterpret_cast<uint4*>(a.hq + (int64_t)g * 128)[l8] = o;
    if (l8 == 0) a.hs[(int64_t)(g % IB) * P + g / IB] = s;
  }
}

// -------------------------------------------------------- down and combine
// A workgroup owns cw columns of Y (a multiple of 4, at most 16 FN, FN
// fragments; chosen so that the CUs' shares are even) and all experts.  A
// unit is 16 MF rows of one expert; the K blocks of all units in a row are
// cut into equal pieces, one for each wave, which streams its piece without a
// pause from one unit to the next.  Cuts fall on granules of G K blocks, at
// most smax to a unit: a piece's sums of a unit go to the place of its first
// granule there, in LDS, so no two waves write the same one.  Then every
// output sums its token's slots in slot order: no atomics, the same bits
// every time.
constexpr int kDownThreads = 64 * kDownWaves;

// The S places of n float4s each into the first, in their order.
template <int S>
__device__ __forceinline__ void join_places(float* lds, int n) {
  v4f* at = reinterpret_cast<v4f*>(lds);
  for (int i = threadIdx.x; i < n; i += kDownThreads) {
    v4f o[S];
#pragma unroll
    for (int s = 0; s < S; ++s) o[s] = at[s * n + i];
#pragma unroll
    for (int s = 1; s < S; ++s) o[0] += o[s];
    at[i] = o[0];
  }
  __syncthreads();
}

// LDSH (few pairs): every workgroup quantises the h of all pairs into LDS
// (rows of I + 16 bytes, so that the 16 rows of a fragment read lie in
// different banks) while its first weights are on their way; else k_moe_quant
// has done it.
template <int MF, int FN, int PF, int OUT, bool LDSH>
__global__ __launch_bounds__(kDownThreads, 2) void k_moe_down(MoeArgs a, int cw, int smax, int most) {
  // smax [P][16 FN] results; units (expert, first row, rows); pos and weight
  // per pair; LDSH: scales [P][I / 128] and codes [P][I + 16]
  extern __shared__ __align__(16) float lds[];
  __shared__ int units_s;   // (not LDSH)
  const int lane = threadIdx.x & 63, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * cw, cols = a.K - n0 < cw ? a.K - n0 : cw;
  const int P = a.T * a.topk, I = a.I, IB = I >> 7;
  int* pos = reinterpret_cast<int*>(lds + smax * P * 16 * FN);
  float* wt = reinterpret_cast<float*>(pos + P);
  uint16_t* ue = reinterpret_cast<uint16_t*>(wt + P);
  uint16_t *ub = ue + P, *un = ub + P;
  float* ls = reinterpret_cast<float*>(pos) + (P * 14 + 15) / 16 * 4;
  int8_t* lq = reinterpret_cast<int8_t*>(ls + (P * IB + 3) / 4 * 4);

  // h of the first groups, 8 lanes to a group (rows behind the last one hold
  // anything, and nobody reads their codes)
  const int l8 = threadIdx.x & 7, g0 = threadIdx.x >> 3;
  constexpr int kPasses = LDSH ? kLdsCodes / 128 / (kDownThreads / 8) : 1;
  float4 raw[kPasses][4];
  if constexpr (LDSH) {
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int g = g0 + k * (kDownThreads / 8);
      if (k * (kDownThreads / 8) >= P * IB) break;
      const float4* at = reinterpret_cast<const float4*>(a.h32 + (int64_t)(g < P * IB ? g : 0) * 128) + l8 * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[k][i] = at[i];
    }
  }

  // the units in the order of the chosen experts.  LDSH: at most 64 experts,
  // one to a lane, in every wave's registers (inc: units up to and with this
  // expert's), so that nothing stands between the tables and the first
  // weights; else a list in LDS, by the first wave
  auto tiles_of = [](int n) { return (n + 16 * MF - 1) / (16 * MF); };
  auto scan = [&](int v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(v, d, 64);
      if (lane >= d) v += o;
    }
    return v;
  };
  int units, n_l = 0, e_l = 0, b_l = 0, inc = 0, pos_l = 0;
  float wt_l = 0.f;
  if constexpr (LDSH) {
    if (lane < most) {
      n_l = a.count[lane];
      e_l = a.expert[lane];
      b_l = a.start[lane];
    }
    if ((int)threadIdx.x < P) {
      pos_l = a.pos[threadIdx.x];
      wt_l = a.weights[threadIdx.x];
    }
    inc = scan(tiles_of(n_l));
    units = __builtin_amdgcn_readlane(inc, 63);
  } else {
    if (wave == 0) {
      int u0 = 0;
      for (int c = 0; c < most; c += 64) {
        const int k = c + lane;
        const int n = k < most ? a.count[k] : 0, e = k < most ? a.expert[k] : 0, b = k < most ? a.start[k] : 0;
        const int t = tiles_of(n), end = scan(t);
        for (int i = 0; i < t; ++i) {
          const int u = u0 + end - t + i;
          ue[u] = (uint16_t)e;
          ub[u] = (uint16_t)(b + i * 16 * MF);
          un[u] = (uint16_t)(n - i * 16 * MF < 16 * MF ? n - i * 16 * MF : 16 * MF);
        }
        u0 += __builtin_amdgcn_readlane(end, 63);
      }
      if (lane == 0) units_s = u0;
    } else {
      for (int p = threadIdx.x - 64; p < P; p += kDownThreads - 64) {
        pos[p] = a.pos[p];
        wt[p] = a.weights[p];
      }
    }
    for (int i = threadIdx.x; i < smax * P * 4 * FN; i += kDownThreads)
      reinterpret_cast<float4*>(lds)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
    units = __builtin_amdgcn_readfirstlane(units_s);
  }
  struct Unit {
    int e, base, rows;
  };
  auto unit = [&](int u) {
    Unit r;
    if constexpr (LDSH) {
      const int k = __ffsll((unsigned long long)__ballot(inc > u)) - 1;
      const int n = __builtin_amdgcn_readlane(n_l, k);
      const int r0 = (u - (__builtin_amdgcn_readlane(inc, k) - tiles_of(n))) * 16 * MF;
      r.e = __builtin_amdgcn_readlane(e_l, k);
      r.base = __builtin_amdgcn_readlane(b_l, k) + r0;
      r.rows = n - r0 < 16 * MF ? n - r0 : 16 * MF;
    } else {
      r.e = __builtin_amdgcn_readfirstlane(ue[u]);
      r.base = __builtin_amdgcn_readfirstlane(ub[u]);
      r.rows = __builtin_amdgcn_readfirstlane(un[u]);
    }
    return r;
  };

  const int G = (IB + smax - 1) / smax, per = (IB + G - 1) / G;   // blocks per granule, granules per unit
  // this workgroup's units, of all the workgroups of its columns
  const int u_lo = (int)((int64_t)units * blockIdx.y / gridDim.y);
  const int u_n = (int)((int64_t)units * (blockIdx.y + 1) / gridDim.y) - u_lo;
  const int lo = u_lo * per + (int)((int64_t)u_n * per * wave / kDownWaves);
  const int hi = u_lo * per + (int)((int64_t)u_n * per * (wave + 1) / kDownWaves);
  // blocks before granule g, counted over the units in a row
  auto blocks_before = [&](int g) { return g / per * IB + (g % per) * G; };
  const int todo = blocks_before(hi) - blocks_before(lo);

  // the unit being loaded and the next block of it
  int lu = lo / per, lkb = lo % per * G;
  rsrc_t rw, rsw, rh, rhs;
  auto open = [&](int u) {
    const Unit c = unit(u);
    rw = rsrc(a.w2 + ((int64_t)c.e * a.K + n0) * I, (int64_t)cols * I);
    rsw = rsrc(a.s2 + (int64_t)c.e * (a.K >> 7) * IB, (int64_t)(a.K >> 7) * IB * 4);
    if (!LDSH) {
      rh = rsrc(a.hq + (int64_t)c.base * I, (int64_t)c.rows * I);
      rhs = rsrc(a.hs + c.base, ((int64_t)(IB - 1) * P + c.rows) * 4);
    }
  };
  const uint32_t off = (uint32_t)((lane & 15) * I + q * 16), soff = (uint32_t)((lane & 15) * 4);
  // the result lane's four columns lie in one 128-row block of the weights
  uint32_t swoff[FN];
#pragma unroll
  for (int f = 0; f < FN; ++f) swoff[f] = (uint32_t)(((n0 + 16 * f + 4 * q) >> 7) * IB * 4);

  v4i wv[PF][FN][2], av[PF][MF][2];
  float sw[PF][FN], sx[PF][MF];
  int left = todo;   // blocks still to load; those past the last read zeros
  auto load = [&](int S) {
    const uint32_t ko = left > 0 ? (uint32_t)lkb * 128u : kOob;
    const uint32_t so = left > 0 ? (uint32_t)lkb * 4u : kOob;
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      wv[S][f][0] = bl16(rw, off + (uint32_t)(16 * f * I) + ko);
      wv[S][f][1] = bl16(rw, off + (uint32_t)(16 * f * I) + ko + 64);
      sw[S][f] = blf(rsw, swoff[f] + so);
    }
    if constexpr (!LDSH) {
#pragma unroll
      for (int j = 0; j < MF; ++j) {
        av[S][j][0] = bl16(rh, off + (uint32_t)(16 * j * I) + ko);
        av[S][j][1] = bl16(rh, off + (uint32_t)(16 * j * I) + ko + 64);
        sx[S][j] = blf(rhs, soff + (uint32_t)(64 * j) + (left > 0 ? so * (uint32_t)P : kOob));
      }
    }
    --left;
    if (++lkb == IB) {
      lkb = 0;
      if (left > 0) open(++lu);
    }
  };
  if (todo > 0) open(lu);
  else rw = rsw = rh = rhs = rsrc(a.w2, 0);
#pragma unroll
  for (int p = 0; p < PF; ++p) {
    load(p);
    __builtin_amdgcn_sched_barrier(0);
  }
  if constexpr (LDSH) {
    if ((int)threadIdx.x < P) {
      pos[threadIdx.x] = pos_l;
      wt[threadIdx.x] = wt_l;
    }
    for (int i = threadIdx.x; i < smax * P * 4 * FN; i += kDownThreads)
      reinterpret_cast<float4*>(lds)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      const int g = g0 + k * (kDownThreads / 8);
      if (k * (kDownThreads / 8) >= P * IB) break;
      float s;
      const uint4 o = quant16(raw[k], &s);
      if (g < P * IB) {
        const int row = g / IB;
        reinterpret_cast<uint4*>(lq + row * (I + 16) + (g - row * IB) * 128)[l8] = o;
        if (l8 == 0) ls[g] = s;
      }
    }
    __syncthreads();
  }

  // the unit being multiplied, its place, and the next block of it
  int u = lo / per, kb = lo % per * G, place = lo % per;
  int base = 0, rows = 0;
  auto take = [&] {
    const Unit c = unit(u);
    base = c.base;
    rows = c.rows;
  };
  if (todo > 0) take();
  v4f acc[FN][MF];
  auto clear = [&] {
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
      for (int j = 0; j < MF; ++j) acc[f][j] = (v4f){0.f, 0.f, 0.f, 0.f};
  };
  clear();
  for (int i = 0; i < todo; i += PF) {
#pragma unroll
    for (int p = 0; p < PF; ++p) {
      if constexpr (LDSH) {
        // a block past the last multiplies zero weights, a row past the last
        // is never stored: both read a valid one
#pragma unroll
        for (int j = 0; j < MF; ++j) {
          const int r = 16 * j + (lane & 15), rc = base + (r < rows ? r : 0);
          const int8_t* at = lq + rc * (I + 16) + kb * 128 + q * 16;
          av[p][j][0] = *reinterpret_cast<const v4i*>(at);
          av[p][j][1] = *reinterpret_cast<const v4i*>(at + 64);
          sx[p][j] = ls[rc * IB + kb];
        }
      }
#pragma unroll
      for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int j = 0; j < MF; ++j)
          acc[f][j] = block_fma(acc[f][j], wv[p][f][0], wv[p][f][1], av[p][j][0], av[p][j][1],
                                __fmul_rn(sx[p][j], sw[p][f]));
      load(p);
      if (i + p < todo && (++kb == IB || i + p + 1 == todo)) {
        float* out = lds + place * P * 16 * FN;
#pragma unroll
        for (int j = 0; j < MF; ++j) {
          const int r = 16 * j + (lane & 15);
#pragma unroll
          for (int f = 0; f < FN; ++f)
            if (r < rows) *reinterpret_cast<v4f*>(out + (base + r) * (16 * FN) + 16 * f + 4 * q) = acc[f][j];
        }
        clear();
        place = kb = 0;
        if (i + p + 1 < todo) {
          ++u;
          take();
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  __syncthreads();
  // the places of each pair's row into the first
  switch (smax) {
    case 2: join_places<2>(lds, P * 4 * FN); break;
    case 4: join_places<4>(lds, P * 4 * FN); break;
    default: break;
  }
  if (gridDim.y > 1) {   // k_moe_combine sums the pairs
    for (int k = wave; k < u_n; k += kDownWaves) {
      const Unit c = unit(u_lo + k);
      for (int i = lane; i < c.rows * cols; i += 64) {
        const int r = i / cols, col = i - r * cols;
        a.out32[(int64_t)(c.base + r) * a.K + n0 + col] = lds[(c.base + r) * 16 * FN + col];
      }
    }
    return;
  }
  for (int i = threadIdx.x; i < a.T * cols; i += kDownThreads) {
    const int t = i / cols, col = i - t * cols;
    float y = 0.f;
    for (int j0 = 0; j0 < a.topk; j0 += 4) {   // four slots' LDS reads at a time
      int r[4];
      float w[4], o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = t * a.topk + (j0 + j < a.topk ? j0 + j : a.topk - 1);
        r[j] = j0 + j < a.topk ? pos[p] : -1;
        w[j] = wt[p];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = lds[(r[j] < 0 ? 0 : r[j]) * 16 * FN + col];
#pragma unroll
      for (int j = 0; j < 4; ++j) y = r[j] < 0 ? y : __builtin_fmaf(w[j], o[j], y);
    }
    const int64_t at = (int64_t)t * a.K + n0 + col;
    if (OUT == OUT_F32)
      static_cast<float*>(a.Y)[at] = y;
    else
      static_cast<uint16_t*>(a.Y)[at] = (uint16_t)f32_to_bf16_rne(y);
  }
}

// Y from the pairs' products, 4 columns per thread, in slot order.
template <int OUT>
__global__ __launch_bounds__(256) void k_moe_combine(MoeArgs a) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= a.T * (a.K >> 2)) return;
  const int t = i / (a.K >> 2), n = (i - t * (a.K >> 2)) * 4;
  float y[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < a.topk; ++j) {
    const int p = t * a.topk + j, r = a.pos[p];
    if (r < 0) continue;
    const float4 o = *reinterpret_cast<const float4*>(a.out32 + (int64_t)r * a.K + n);
    const float w = a.weights[p];
    y[0] = __builtin_fmaf(w, o.x, y[0]);
    y[1] = __builtin_fmaf(w, o.y, y[1]);
    y[2] = __builtin_fmaf(w, o.z, y[2]);
    y[3] = __builtin_fmaf(w, o.w, y[3]);
  }
  const int64_t at = (int64_t)t * a.K + n;
  if (OUT == OUT_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(a.Y) + at) = make_float4(y[0], y[1], y[2], y[3]);
  } else {
    uint2 o;
    o.x = f32_to_bf16_rne(y[0]) | (f32_to_bf16_rne(y[1]) << 16);
    o.y = f32_to_bf16_rne(y[2]) | (f32_to_bf16_rne(y[3]) << 16);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.Y) + at) = o;
  }
}

template <int MF, int FN, int PF, bool LDSH>
hipError_t down_launch(const MoeArgs& a, const MoePlan& p, OutKind out, hipStream_t st) {
  const dim3 grid((unsigned)((a.K + p.cw - 1) / p.cw), (unsigned)p.z), block(kDownThreads);
  if (out == OUT_F32)
    hipLaunchKernelGGL((k_moe_down<MF, FN, PF, OUT_F32, LDSH>), grid, block, p.down_lds, st, a, p.cw, p.smax, p.most);
  else
    hipLaunchKernelGGL((k_moe_down<MF, FN, PF, OUT_BF16, LDSH>), grid, block, p.down_lds, st, a, p.cw, p.smax, p.most);
  return hipGetLastError();
}

template <int MFBIG, int FC, int WK>
hipError_t gate_up_launch(const MoeArgs& a, const MoePlan& p, hipStream_t st) {
  const int cols = 16 * FC * (kGuWaves / WK);
  hipLaunchKernelGGL((k_moe_gate_up<MFBIG, FC, WK>), dim3((unsigned)(a.I / cols), (unsigned)p.most), dim3(kGuThreads),
                     p.gu_lds, st, a);
  return hipGetLastError();
}

}  // namespace

// Workspace: h (fp32), its codes and their scales, a row per pair; each
// pair's row; the chosen experts' indices, rows and first rows; the pairs'
// products where several workgroups share the columns.
int64_t moe_workspace(int64_t T, int64_t topk, int64_t I, int64_t K, MoeArgs* a, void* ws) {
  const int64_t P = T * topk;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(ws) + (uintptr_t)at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  MoeArgs m = a ? *a : MoeArgs();
  const bool in_down = moe_quant_in_down(P, I);
  m.h32 = reinterpret_cast<float*>(take(P * I * 4));
  m.hq = reinterpret_cast<int8_t*>(take(in_down ? 0 : P * I));
  m.hs = reinterpret_cast<float*>(take(in_down ? 0 : P * (I / 128) * 4));
  m.pos = reinterpret_cast<int32_t*>(take(P * 4));
  m.expert = reinterpret_cast<int32_t*>(take(P * 4));
  m.count = reinterpret_cast<int32_t*>(take(P * 4));
  m.start = reinterpret_cast<int32_t*>(take(P * 4));
  m.out32 = reinterpret_cast<float*>(take(in_down || K > kSplitMaxK ? 0 : P * K * 4));
  if (a) *a = m;
  return at;
}

hipError_t launch_moe_block(const MoeArgs& a, OutKind out, hipStream_t st) {
  const MoePlan p = moe_plan(a.T, a.topk, a.E, a.I, a.K);
  hipError_t e = p.gu_mf == 4   ? gate_up_launch<4, 2, 4>(a, p, st)
                 : p.gu_wk == 2 ? gate_up_launch<2, 2, 2>(a, p, st)
                 : p.gu_fc == 1 ? gate_up_launch<2, 1, 4>(a, p, st)
                                : gate_up_launch<2, 2, 4>(a, p, st);
  if (e != hipSuccess) return e;
  const bool one = p.down_fn == 1;   // one fragment of columns
  if (p.in_down) return one ? down_launch<1, 1, 8, true>(a, p, out, st) : down_launch<1, 2, 6, true>(a, p, out, st);
  const int P = a.T * a.topk, IB = a.I / 128;
  hipLaunchKernelGGL(k_moe_quant, dim3((unsigned)((P * IB + 31) / 32)), dim3(256), 0, st, a, P, IB);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.down_mf == 1)
    e = one ? down_launch<1, 1, 8, false>(a, p, out, st) : down_launch<1, 2, 6, false>(a, p, out, st);
  else if (p.down_mf == 2)
    e = one ? down_launch<2, 1, 6, false>(a, p, out, st) : down_launch<2, 2, 4, false>(a, p, out, st);
  else
    e = one ? down_launch<4, 1, 3, false>(a, p, out, st) : down_launch<4, 2, 3, false>(a, p, out, st);
  if (e != hipSuccess || p.z == 1) return e;
  const dim3 grid((unsigned)(((int64_t)a.T * (a.K / 4) + 255) / 256));
  if (out == OUT_F32)
    hipLaunchKernelGGL((k_moe_combine<OUT_F32>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((k_moe_combine<OUT_BF16>), grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace w8
