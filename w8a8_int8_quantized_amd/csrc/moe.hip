// A whole mixture-of-experts layer for a few tokens, in two kernels (gfx950).
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
// (3 I K bytes for each expert that a token chose), so both kernels stream
// them once, straight from global memory into MFMA operand registers.  A
// "pair" is one slot of one token (t, j), p = t topk + j; the pairs of one
// expert are the rows of its products, in the order of p, and the rows of all
// experts in the order of the expert index are the rows of hq.  A pair whose
// id is outside 0 .. E - 1 has no row.
#include <type_traits>

#include "common.h"
#include "launch.h"

namespace w8 {
namespace {

constexpr int kMaxPairs = 1024;
template <int N>
using Int = std::integral_constant<int, N>;
typedef __amdgpu_buffer_rsrc_t rsrc_t;

// Added to the offset of a load that must read zero: beyond the range of
// every descriptor here (at most 1024 rows x 2^17 bytes), twice it still
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
// expert e against its gate columns c0 .. c0 + 15 (acc[0]) and the up columns
// of the same index (acc[1]).  PF blocks of loads stay in flight in a
// register ring.
template <int MF, int PF, int WK>
__device__ __forceinline__ void gate_up_sums(const MoeArgs& a, int e, int c0, int par, int r0, int n,
                                             const uint16_t* tok, v4f (&acc)[2][MF]) {
  const int lane = threadIdx.x & 63;
  const int q = lane >> 4;
  const int K = a.K, KB = K >> 7;
  const int64_t wrow = (int64_t)e * 2 * a.I + c0;
  const int64_t srow = (int64_t)e * 2 * (a.I >> 7) + (c0 >> 7);
  const rsrc_t rg = rsrc(a.w13 + wrow * K, (int64_t)16 * K);
  const rsrc_t ru = rsrc(a.w13 + (wrow + a.I) * K, (int64_t)16 * K);
  const rsrc_t rsg = rsrc(a.s13 + srow * KB, (int64_t)KB * 4);
  const rsrc_t rsu = rsrc(a.s13 + (srow + (a.I >> 7)) * KB, (int64_t)KB * 4);
  const rsrc_t ra = rsrc(a.A, (int64_t)a.T * K);
  const rsrc_t rsa = rsrc(a.sa, (int64_t)a.T * KB * 4);
  const uint32_t woff = (uint32_t)((lane & 15) * K + q * 16);
  uint32_t aoff[MF], saoff[MF];
#pragma unroll
  for (int j = 0; j < MF; ++j) {
    const int r = r0 + 16 * j + (lane & 15);
    const uint32_t t = r < n ? tok[r] : 0u;
    aoff[j] = r < n ? t * (uint32_t)K + q * 16 : kOob;
    saoff[j] = r < n ? t * (uint32_t)KB * 4u : kOob;
  }
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int j = 0; j < MF; ++j) acc[f][j] = (v4f){0.f, 0.f, 0.f, 0.f};

  v4i wv[PF][2][2], av[PF][MF][2];
  float sw[PF][2], sx[PF][MF];
  auto load = [&](int P, int kb) {
    const uint32_t ko = kb < KB ? (uint32_t)kb * 128u : kOob;
    const uint32_t so = kb < KB ? (uint32_t)kb * 4u : kOob;
    wv[P][0][0] = bl16(rg, woff + ko);
    wv[P][0][1] = bl16(rg, woff + ko + 64);
    wv[P][1][0] = bl16(ru, woff + ko);
    wv[P][1][1] = bl16(ru, woff + ko + 64);
    sw[P][0] = blf(rsg, so);
    sw[P][1] = blf(rsu, so);
#pragma unroll
    for (int j = 0; j < MF; ++j) {
      av[P][j][0] = bl16(ra, aoff[j] + ko);
      av[P][j][1] = bl16(ra, aoff[j] + ko + 64);
      sx[P][j] = blf(rsa, saoff[j] + so);
    }
  };
#pragma unroll
  for (int p = 0; p < PF; ++p) {
    load(p, par + WK * p);
    __builtin_amdgcn_sched_barrier(0);
  }
  // blocks past the last hold zeros
  for (int kb = par; kb < KB; kb += WK * PF) {
#pragma unroll
    for (int p = 0; p < PF; ++p) {
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int j = 0; j < MF; ++j)
          acc[f][j] = block_fma(acc[f][j], wv[p][f][0], wv[p][f][1], av[p][j][0], av[p][j][1],
                                __fmul_rn(sx[p][j], sw[p][f]));
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
__device__ __forceinline__ uint4 quant16(float* v, float* scale) {
  const QScale sc = make_scale(max8(amax_n(v, 16)));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = quant_one(v[i], sc);
  *scale = sc.s;
  return make_uint4(pack4(v[0], v[1], v[2], v[3]), pack4(v[4], v[5], v[6], v[7]), pack4(v[8], v[9], v[10], v[11]),
                    pack4(v[12], v[13], v[14], v[15]));
}

// ---------------------------------------------------- who has which expert
constexpr int kGuWaves = 4, kGuThreads = 64 * kGuWaves;
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

// Grid (I / 16, min(pairs, E)): 16 columns of h of one expert per workgroup,
// whose four waves split the K blocks.  A workgroup this small keeps the load
// of the CUs even: each CU streams at a rate of its own (its outstanding
// loads over the memory's latency), so the kernel takes as long as the CU
// with the most bytes.  The 128 columns of a quantisation group lie in eight
// workgroups; h leaves in fp32 and is quantised by its readers.
template <int MF, int PF>
__device__ __forceinline__ void gate_up_rows(const MoeArgs& a, const Chosen& c, int r0, const uint16_t* tok,
                                             float* lds) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tile = blockIdx.x;
  v4f acc[2][MF];
  gate_up_sums<MF, PF, kGuWaves>(a, c.e, tile * 16, wave, r0, c.n, tok, acc);
  v4f* red = reinterpret_cast<v4f*>(lds);
  if (wave > 0) {
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int j = 0; j < MF; ++j) red[(((wave - 1) * 2 + f) * MF + j) * 64 + lane] = acc[f][j];
  }
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int j = 0; j < MF; ++j) {
#pragma unroll
      for (int w = 0; w < kGuWaves - 1; ++w) {
        acc[0][j] += red[((w * 2 + 0) * MF + j) * 64 + lane];
        acc[1][j] += red[((w * 2 + 1) * MF + j) * 64 + lane];
      }
      const int r = r0 + 16 * j + (lane & 15);
      if (r < c.n)
        *reinterpret_cast<v4f*>(a.h32 + (int64_t)(c.base + r) * a.I + tile * 16 + 4 * (lane >> 4)) =
            silu_mul(acc[0][j], acc[1][j]);
    }
  }
  __syncthreads();
}

template <int MFMAX>
__global__ __launch_bounds__(kGuThreads, 4) void k_moe_gate_up(MoeArgs a) {
  __shared__ uint16_t tok[kMaxPairs];
  extern __shared__ float lds[];   // E ints, then the waves' sums
  const Chosen c = choose(a, blockIdx.y, blockIdx.x == 0, reinterpret_cast<int*>(lds), tok);
  if (c.e < 0) return;
  // a token that names an expert twice gives it two rows, so n can pass T:
  // the rows past 16 MFMAX take further passes over the weights
  auto rows = [&](auto mf, auto pf) {
    for (int r0 = 0; r0 < c.n; r0 += 16 * mf()) gate_up_rows<mf(), pf()>(a, c, r0, tok, lds);
  };
  if (MFMAX == 1 || c.n <= 16) rows(Int<1>(), Int<3>());
  else if (MFMAX == 2 || c.n <= 32) rows(Int<MFMAX < 2 ? MFMAX : 2>(), Int<2>());
  else rows(Int<MFMAX>(), Int<1>());
}

// The codes and scales of h, a group per 8 lanes; rows behind the last pair's
// hold whatever the workspace held and nobody reads theirs.
__global__ __launch_bounds__(256) void k_moe_quant(MoeArgs a, int groups) {
  const int g = blockIdx.x * 32 + (threadIdx.x >> 3), l8 = threadIdx.x & 7;
  const float4* at = reinterpret_cast<const float4*>(a.h32 + (int64_t)(g < groups ? g : groups - 1) * 128) + l8 * 4;
  float v[16], s;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 x = at[i];
    v[4 * i] = x.x;
    v[4 * i + 1] = x.y;
    v[4 * i + 2] = x.z;
    v[4 * i + 3] = x.w;
  }
  const uint4 o = quant16(v, &s);
  if (g < groups) {
    reinterpret_cast<uint4*>(a.hq + (int64_t)g * 128)[l8] = o;
    if (l8 == 0) a.hs[g] = s;
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
constexpr int kDownWaves = 8, kDownThreads = 64 * kDownWaves;

// LDSH (few pairs): every workgroup quantises the h of all pairs into LDS
// (rows of I + 16 bytes, so that the 16 rows of a fragment read lie in
// different banks) while its first weights are on their way; else k_moe_quant
// has done it.
template <int MF, int FN, int PF, int OUT, bool LDSH>
__global__ __launch_bounds__(kDownThreads, 2) void k_moe_down(MoeArgs a, int cw, int smax, int most) {
  // smax [P][16 FN] results; units (expert, first row, rows); pos and weight
  // per pair; LDSH: scales [P][I / 128] and codes [P][I + 16]
  extern __shared__ float lds[];
  __shared__ int units_s;
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
  float4 raw[4];
  auto fetch = [&](int g) {
    const float4* at = reinterpret_cast<const float4*>(a.h32 + (int64_t)(g < P * IB ? g : 0) * 128) + l8 * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i] = at[i];
  };
  if (LDSH) fetch(g0);

  // the list of units, by the first wave; pos and weights, by the others
  if (wave == 0) {
    int units = 0;
    for (int c = 0; c < most; c += 64) {
      const int k = c + lane;
      const int n = k < most ? a.count[k] : 0, e = k < most ? a.expert[k] : 0, b = k < most ? a.start[k] : 0;
      const int tiles = (n + 16 * MF - 1) / (16 * MF);
      int inc = tiles;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(inc, d, 64);
        if (lane >= d) inc += v;
      }
      for (int i = 0; i < tiles; ++i) {
        const int u = units + inc - tiles + i;
        ue[u] = (uint16_t)e;
        ub[u] = (uint16_t)(b + i * 16 * MF);
        un[u] = (uint16_t)(n - i * 16 * MF < 16 * MF ? n - i * 16 * MF : 16 * MF);
      }
      units += __builtin_amdgcn_readlane(inc, 63);
    }
    if (lane == 0) units_s = units;
  } else {
    for (int p = threadIdx.x - 64; p < P; p += kDownThreads - 64) {
      pos[p] = a.pos[p];
      wt[p] = a.weights[p];
    }
  }
  for (int i = threadIdx.x; i < smax * P * 4 * FN; i += kDownThreads)
    reinterpret_cast<float4*>(lds)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
  const int units = __builtin_amdgcn_readfirstlane(units_s);

  const int G = (IB + smax - 1) / smax, per = (IB + G - 1) / G;   // blocks per granule, granules per unit
  const int lo = (int)((int64_t)units * per * wave / kDownWaves);
  const int hi = (int)((int64_t)units * per * (wave + 1) / kDownWaves);
  // blocks before granule g, counted over the units in a row
  auto blocks_before = [&](int g) { return g / per * IB + (g % per) * G; };
  const int todo = blocks_before(hi) - blocks_before(lo);

  // the unit being loaded and the next block of it
  int lu = lo / per, lkb = lo % per * G;
  rsrc_t rw, rsw, rh, rhs;
  int lbase = 0, lrows = 0;
  auto open = [&](int u) {
    const int e = __builtin_amdgcn_readfirstlane(ue[u]);
    lbase = __builtin_amdgcn_readfirstlane(ub[u]);
    lrows = __builtin_amdgcn_readfirstlane(un[u]);
    rw = rsrc(a.w2 + ((int64_t)e * a.K + n0) * I, (int64_t)cols * I);
    rsw = rsrc(a.s2 + (int64_t)e * (a.K >> 7) * IB, (int64_t)(a.K >> 7) * IB * 4);
    if (!LDSH) {
      rh = rsrc(a.hq + (int64_t)lbase * I, (int64_t)lrows * I);
      rhs = rsrc(a.hs + (int64_t)lbase * IB, (int64_t)lrows * IB * 4);
    }
  };
  const uint32_t off = (uint32_t)((lane & 15) * I + q * 16), soff = (uint32_t)((lane & 15) * IB * 4);
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
        sx[S][j] = blf(rhs, soff + (uint32_t)(16 * j * IB * 4) + so);
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
    for (int g = g0; g - g0 < P * IB; g += kDownThreads / 8) {
      if (g != g0) fetch(g);
      float v[16], s;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[4 * i] = raw[i].x;
        v[4 * i + 1] = raw[i].y;
        v[4 * i + 2] = raw[i].z;
        v[4 * i + 3] = raw[i].w;
      }
      const uint4 o = quant16(v, &s);
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
    base = __builtin_amdgcn_readfirstlane(ub[u]);
    rows = __builtin_amdgcn_readfirstlane(un[u]);
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
  for (int i = threadIdx.x; i < a.T * cols; i += kDownThreads) {
    const int t = i / cols, col = i - t * cols;
    float y = 0.f;
    for (int j = 0; j < a.topk; ++j) {
      const int p = t * a.topk + j, r = pos[p];
      if (r < 0) continue;
      float o = lds[r * 16 * FN + col];
      for (int s = 1; s < smax; ++s) o += lds[(s * P + r) * 16 * FN + col];
      y = __builtin_fmaf(wt[p], o, y);
    }
    const int64_t at = (int64_t)t * a.K + n0 + col;
    if (OUT == OUT_F32)
      static_cast<float*>(a.Y)[at] = y;
    else
      static_cast<uint16_t*>(a.Y)[at] = (uint16_t)f32_to_bf16_rne(y);
  }
}

// Pairs whose h every down workgroup quantises for itself, at most.
constexpr int64_t kLdsPairs = 64, kLdsCodes = 32768;

bool quant_in_down(int64_t P, int64_t I) { return P <= kLdsPairs && P * I <= kLdsCodes; }

// Columns per down workgroup: a multiple of 4 up to 32, the widest of those
// that give the fullest CU the fewest columns.
int down_columns(int K) {
  int best = 16, most = 1 << 30;
  for (int cw = 32; cw >= 4; cw -= 4) {
    const int wgs = (K + cw - 1) / cw, load = (wgs + 255) / 256 * cw;
    if (load < most) {
      most = load;
      best = cw;
    }
  }
  return best;
}

template <int MF, int FN, int PF, bool LDSH>
hipError_t down_launch(const MoeArgs& a, OutKind out, int cw, int most, hipStream_t st) {
  const int P = a.T * a.topk, IB = a.I / 128;
  const size_t res = (size_t)P * FN * 64;
  const size_t rest = (size_t)(P * 14 + 15) / 16 * 16 +
                      (LDSH ? (size_t)(P * IB + 3) / 4 * 16 + (size_t)P * (a.I + 16) : 0);
  int smax = 1;
  while (smax * 2 <= IB && smax * 2 <= kDownWaves && smax * 2 * res + rest <= 131072) smax *= 2;
  const dim3 grid((unsigned)((a.K + cw - 1) / cw)), block(kDownThreads);
  const size_t lds = smax * res + rest;
  if (out == OUT_F32)
    hipLaunchKernelGGL((k_moe_down<MF, FN, PF, OUT_F32, LDSH>), grid, block, lds, st, a, cw, smax, most);
  else
    hipLaunchKernelGGL((k_moe_down<MF, FN, PF, OUT_BF16, LDSH>), grid, block, lds, st, a, cw, smax, most);
  return hipGetLastError();
}

template <int MFMAX>
hipError_t gate_up_launch(const MoeArgs& a, int most, hipStream_t st) {
  const size_t sums = (size_t)(kGuWaves - 1) * 2 * MFMAX * 1024, owner = (size_t)a.E * 4;
  hipLaunchKernelGGL((k_moe_gate_up<MFMAX>), dim3((unsigned)(a.I / 16), (unsigned)most), dim3(kGuThreads),
                     sums > owner ? sums : owner, st, a);
  return hipGetLastError();
}

}  // namespace

// Workspace: h (fp32), its codes and their scales, a row per pair; each
// pair's row; the chosen experts' indices, rows and first rows.
int64_t moe_workspace(int64_t T, int64_t topk, int64_t I, MoeArgs* a, void* ws) {
  const int64_t P = T * topk;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    char* p = static_cast<char*>(ws) + at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  MoeArgs m = a ? *a : MoeArgs();
  const bool in_down = quant_in_down(P, I);
  m.h32 = reinterpret_cast<float*>(take(P * I * 4));
  m.hq = reinterpret_cast<int8_t*>(take(in_down ? 0 : P * I));
  m.hs = reinterpret_cast<float*>(take(in_down ? 0 : P * (I / 128) * 4));
  m.pos = reinterpret_cast<int32_t*>(take(P * 4));
  m.expert = reinterpret_cast<int32_t*>(take(P * 4));
  m.count = reinterpret_cast<int32_t*>(take(P * 4));
  m.start = reinterpret_cast<int32_t*>(take(P * 4));
  if (a) *a = m;
  return at;
}

hipError_t launch_moe_block(const MoeArgs& a, OutKind out, hipStream_t st) {
  const int P = a.T * a.topk, IB = a.I / 128;
  const int most = P < a.E ? P : a.E;   // chosen experts, at most
  hipError_t e = a.T <= 16   ? gate_up_launch<1>(a, most, st)
                 : a.T <= 32 ? gate_up_launch<2>(a, most, st)
                             : gate_up_launch<4>(a, most, st);
  if (e != hipSuccess) return e;
  const int cw = down_columns(a.K);
  if (quant_in_down(P, a.I))
    return cw <= 16 ? down_launch<1, 1, 8, true>(a, out, cw, most, st)
                    : down_launch<1, 2, 6, true>(a, out, cw, most, st);
  hipLaunchKernelGGL(k_moe_quant, dim3((unsigned)((P * IB + 31) / 32)), dim3(256), 0, st, a, P * IB);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  // rows per unit by the mean rows of an expert (a unit of more rows than its
  // expert has costs registers, one of fewer reads the weights again)
  if (P <= 12 * a.E)
    return cw <= 16 ? down_launch<1, 1, 8, false>(a, out, cw, most, st)
                    : down_launch<1, 2, 6, false>(a, out, cw, most, st);
  return cw <= 16 ? down_launch<4, 1, 3, false>(a, out, cw, most, st)
                  : down_launch<4, 2, 3, false>(a, out, cw, most, st);
}

}  // namespace w8
