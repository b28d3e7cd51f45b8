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
#include "common.h"
#include "launch.h"

namespace w8 {
namespace {

constexpr int kMaxPairs = 1024;
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
// A workgroup owns one quantisation group of h: 128 columns, 128 gate and 128
// up rows of W_gate_up, of one expert.  Wave w takes columns 16 (w & 7) .. +15
// of both and the K blocks of parity w >> 3; the two parities' sums are added
// through LDS.  Fragment layout (v_mfma_i32_16x16x64_i8, weights as operand
// A): lane l holds weight row l & 15 and activation row l & 15, bytes
// 16 (l >> 4) .. +15 of each 64-wide half of the K block; the result lane
// holds columns 4 (l >> 4) .. +3 of activation row l & 15.
constexpr int kGuWaves = 16;
constexpr int kHs = 132;   // floats between the rows of the h tile in LDS

template <int MF, int PF>
__device__ __forceinline__ void gate_up_rows(const MoeArgs& a, int e, int g, int base, int r0, int n,
                                             const uint16_t* tok, float* lds) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, col = wave & 7, par = wave >> 3;
  const int K = a.K, KB = K >> 7;
  const int64_t wrow = (int64_t)e * 2 * a.I + g * 128 + col * 16;
  const int64_t srow = (int64_t)e * 2 * (a.I >> 7) + g;
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
  v4f acc[2][MF];
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
    load(p, par + 2 * p);
    __builtin_amdgcn_sched_barrier(0);
  }
  // blocks past the last hold zeros
  for (int kb = par; kb < KB; kb += 2 * PF) {
#pragma unroll
    for (int p = 0; p < PF; ++p) {
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int j = 0; j < MF; ++j)
          acc[f][j] = block_fma(acc[f][j], wv[p][f][0], wv[p][f][1], av[p][j][0], av[p][j][1],
                                __fmul_rn(sx[p][j], sw[p][f]));
      load(p, kb + 2 * (p + PF));
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // the odd blocks' sums through LDS, then h into LDS as [16 MF][128]
  v4f* red = reinterpret_cast<v4f*>(lds);
  if (par == 1) {
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int j = 0; j < MF; ++j) red[((col * 2 + f) * MF + j) * 64 + lane] = acc[f][j];
  }
  __syncthreads();
  if (par == 0) {
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int j = 0; j < MF; ++j) acc[f][j] += red[((col * 2 + f) * MF + j) * 64 + lane];
  }
  __syncthreads();
  if (par == 0) {
#pragma unroll
    for (int j = 0; j < MF; ++j) {
      v4f h;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float x = acc[0][j][r];
        h[r] = x / (1.0f + expf(-x)) * acc[1][j][r];
      }
      *reinterpret_cast<v4f*>(lds + (16 * j + (lane & 15)) * kHs + col * 16 + 4 * q) = h;
    }
  }
  __syncthreads();
  // the group quantiser, 8 lanes per row; h is quantised from fp32 (a 16-bit
  // h would be written by nobody and read by nobody)
  const int row = threadIdx.x >> 3, l8 = threadIdx.x & 7;
  if (row < 16 * MF && r0 + row < n) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = lds[row * kHs + l8 * 16 + i];
    const QScale sc = make_scale(max8(amax_n(v, 16)));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = quant_one(v[i], sc);
    uint4 o;
    o.x = pack4(v[0], v[1], v[2], v[3]);
    o.y = pack4(v[4], v[5], v[6], v[7]);
    o.z = pack4(v[8], v[9], v[10], v[11]);
    o.w = pack4(v[12], v[13], v[14], v[15]);
    const int64_t hr = base + r0 + row;
    reinterpret_cast<uint4*>(a.hq + hr * a.I + g * 128)[l8] = o;
    if (l8 == 0) a.hs[hr * (a.I >> 7) + g] = sc.s;
  }
  __syncthreads();   // lds is free for the next rows
}

// Grid (I / 128, pairs).  The workgroups of the first pair of an expert do
// that expert's rows, the others leave.
template <int MFMAX>
__global__ __launch_bounds__(64 * kGuWaves) void k_moe_gate_up(MoeArgs a) {
  __shared__ uint16_t tok[kMaxPairs];
  extern __shared__ float lds[];
  const int lane = threadIdx.x & 63;
  const int p = blockIdx.y, g = blockIdx.x;
  const int P = a.T * a.topk;
  const int e = __builtin_amdgcn_readfirstlane(a.ids[p]);
  const bool valid = e >= 0 && e < a.E;
  // rows of this expert, its first pair, the pairs of lower experts before it
  int n = 0, base = 0, first = P, rank = 0;
  if (valid) {
    for (int c = 0; c < P; c += 64) {
      const int i = c + lane;
      const int id = i < P ? a.ids[i] : -1;
      const uint64_t m = __ballot(id == e);
      base += __popcll(__ballot(id >= 0 && id < e));
      if (m && first == P) first = c + __ffsll((unsigned long long)m) - 1;
      if (c + 64 <= p) rank += __popcll(m);
      else if (c <= p) rank += __popcll(m & ((1ull << (p - c)) - 1));
      if (first == p && id == e && threadIdx.x < 64)
        tok[n + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)(i / a.topk);
      n += __popcll(m);
    }
  }
  if (g == 0 && threadIdx.x == 0) {
    a.pos[p] = valid ? base + rank : -1;
    a.count[p] = valid && first == p ? n : 0;
    a.start[p] = base;
  }
  if (!valid || first != p) return;
  __syncthreads();
  // a token that names an expert twice gives it two rows, so n can pass T:
  // the rows past 16 MFMAX take further passes over the weights
  if (MFMAX == 1 || n <= 16) {
    for (int r0 = 0; r0 < n; r0 += 16) gate_up_rows<1, 3>(a, e, g, base, r0, n, tok, lds);
  } else if (MFMAX == 2 || n <= 32) {
    if constexpr (MFMAX >= 2)
      for (int r0 = 0; r0 < n; r0 += 32) gate_up_rows<2, 2>(a, e, g, base, r0, n, tok, lds);
  } else {
    if constexpr (MFMAX >= 4)
      for (int r0 = 0; r0 < n; r0 += 64) gate_up_rows<4, 2>(a, e, g, base, r0, n, tok, lds);
  }
}

// -------------------------------------------------------- down and combine
// A workgroup owns 16 columns of Y and all experts: a unit is one expert's K
// blocks s, s + S, ... and the waves take the units in turn.  Each unit's
// rows go to their own place in LDS (no two units write the same one), then
// every output sums its token's slots in slot order: no atomics, the same
// bits every time.
constexpr int kDownWaves = 8;

template <int MF, int PF>
__device__ __forceinline__ void down_rows(const MoeArgs& a, int e, int base, int n, int r0, int n0, int s, int S,
                                          float* out) {
  const int lane = threadIdx.x & 63;
  const int q = lane >> 4;
  const int I = a.I, IB = I >> 7;
  const rsrc_t rw = rsrc(a.w2 + ((int64_t)e * a.K + n0) * I, (int64_t)16 * I);
  const rsrc_t rsw = rsrc(a.s2 + ((int64_t)e * (a.K >> 7) + (n0 >> 7)) * IB, (int64_t)IB * 4);
  const rsrc_t rh = rsrc(a.hq + (int64_t)(base + r0) * I, (int64_t)(n - r0) * I);
  const rsrc_t rhs = rsrc(a.hs + (int64_t)(base + r0) * IB, (int64_t)(n - r0) * IB * 4);
  const uint32_t off = (uint32_t)((lane & 15) * I + q * 16), soff = (uint32_t)((lane & 15) * IB * 4);
  v4f acc[MF];
#pragma unroll
  for (int j = 0; j < MF; ++j) acc[j] = (v4f){0.f, 0.f, 0.f, 0.f};
  v4i wv[PF][2], av[PF][MF][2];
  float sw[PF], sx[PF][MF];
  auto load = [&](int P, int kb) {
    const uint32_t ko = kb < IB ? (uint32_t)kb * 128u : kOob;
    const uint32_t so = kb < IB ? (uint32_t)kb * 4u : kOob;
    wv[P][0] = bl16(rw, off + ko);
    wv[P][1] = bl16(rw, off + ko + 64);
    sw[P] = blf(rsw, so);
#pragma unroll
    for (int j = 0; j < MF; ++j) {
      av[P][j][0] = bl16(rh, off + (uint32_t)(16 * j * I) + ko);
      av[P][j][1] = bl16(rh, off + (uint32_t)(16 * j * I) + ko + 64);
      sx[P][j] = blf(rhs, soff + (uint32_t)(16 * j * IB * 4) + so);
    }
  };
#pragma unroll
  for (int p = 0; p < PF; ++p) {
    load(p, s + S * p);
    __builtin_amdgcn_sched_barrier(0);
  }
  for (int kb = s; kb < IB; kb += S * PF) {
#pragma unroll
    for (int p = 0; p < PF; ++p) {
#pragma unroll
      for (int j = 0; j < MF; ++j)
        acc[j] = block_fma(acc[j], wv[p][0], wv[p][1], av[p][j][0], av[p][j][1], __fmul_rn(sx[p][j], sw[p]));
      load(p, kb + S * (p + PF));
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int j = 0; j < MF; ++j) {
    const int r = r0 + 16 * j + (lane & 15);
    if (r < n) *reinterpret_cast<v4f*>(out + (base + r) * 16 + 4 * q) = acc[j];
  }
}

template <int MFMAX, int OUT>
__global__ __launch_bounds__(64 * kDownWaves) void k_moe_down(MoeArgs a, int S) {
  __shared__ uint16_t list[kMaxPairs];
  extern __shared__ float lds[];   // S times one [rows][16] array
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16;
  const int P = a.T * a.topk;
  int active = 0;
  for (int c = 0; c < P; c += 64) {
    const bool has = c + lane < P && a.count[c + lane] > 0;
    const uint64_t m = __ballot(has);
    if (has && wave == 0) list[active + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)(c + lane);
    active += __popcll(m);
  }
  __syncthreads();
  for (int u = wave; u < active * S; u += kDownWaves) {
    const int p = __builtin_amdgcn_readfirstlane(list[u / S]), s = u % S;
    const int e = __builtin_amdgcn_readfirstlane(a.ids[p]), n = __builtin_amdgcn_readfirstlane(a.count[p]);
    const int base = __builtin_amdgcn_readfirstlane(a.start[p]);
    float* out = lds + (int64_t)s * P * 16;
    if (MFMAX == 1 || n <= 16) {
      for (int r0 = 0; r0 < n; r0 += 16) down_rows<1, 4>(a, e, base, n, r0, n0, s, S, out);
    } else if (MFMAX == 2 || n <= 32) {
      if constexpr (MFMAX >= 2)
        for (int r0 = 0; r0 < n; r0 += 32) down_rows<2, 4>(a, e, base, n, r0, n0, s, S, out);
    } else {
      if constexpr (MFMAX >= 4)
        for (int r0 = 0; r0 < n; r0 += 64) down_rows<4, 2>(a, e, base, n, r0, n0, s, S, out);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * 16; i += 64 * kDownWaves) {
    const int t = i >> 4, c = i & 15;
    float y = 0.f;
    for (int j = 0; j < a.topk; ++j) {
      const int p = t * a.topk + j, r = a.pos[p];
      if (r < 0) continue;
      float o = lds[r * 16 + c];
      for (int s = 1; s < S; ++s) o += lds[((int64_t)s * P + r) * 16 + c];
      y = __builtin_fmaf(a.weights[p], o, y);
    }
    const int64_t at = (int64_t)t * a.K + n0 + c;
    if (OUT == OUT_F32)
      static_cast<float*>(a.Y)[at] = y;
    else
      static_cast<uint16_t*>(a.Y)[at] = (uint16_t)f32_to_bf16_rne(y);
  }
}

template <int MFMAX>
hipError_t moe_launch(const MoeArgs& a, OutKind out, hipStream_t st) {
  const int P = a.T * a.topk;
  hipLaunchKernelGGL((k_moe_gate_up<MFMAX>), dim3((unsigned)(a.I / 128), (unsigned)P), dim3(64 * kGuWaves),
                     MFMAX * 16384, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // few experts: several waves share an expert's K blocks
  int S = 1;
  while (S * 2 * P <= 2 * kDownWaves && S * 2 <= a.I / 128) S *= 2;
  const dim3 grid((unsigned)(a.K / 16)), block(64 * kDownWaves);
  const size_t lds = (size_t)S * P * 64;
  if (out == OUT_F32)
    hipLaunchKernelGGL((k_moe_down<MFMAX, OUT_F32>), grid, block, lds, st, a, S);
  else
    hipLaunchKernelGGL((k_moe_down<MFMAX, OUT_BF16>), grid, block, lds, st, a, S);
  return hipGetLastError();
}

}  // namespace

// Workspace: the codes of h, their scales, and three int32 per pair.
int64_t moe_workspace(int64_t T, int64_t topk, int64_t I, MoeArgs* a, void* ws) {
  const int64_t P = T * topk;
  auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
  const int64_t scales = up(P * I), pos = scales + up(P * (I / 128) * 4), count = pos + up(P * 4),
                start = count + up(P * 4);
  if (a) {
    char* b = static_cast<char*>(ws);
    a->hq = reinterpret_cast<int8_t*>(b);
    a->hs = reinterpret_cast<float*>(b + scales);
    a->pos = reinterpret_cast<int32_t*>(b + pos);
    a->count = reinterpret_cast<int32_t*>(b + count);
    a->start = reinterpret_cast<int32_t*>(b + start);
  }
  return start + up(P * 4);
}

hipError_t launch_moe_block(const MoeArgs& a, OutKind out, hipStream_t st) {
  if (a.T <= 16) return moe_launch<1>(a, out, st);
  if (a.T <= 32) return moe_launch<2>(a, out, st);
  return moe_launch<4>(a, out, st);
}

}  // namespace w8
