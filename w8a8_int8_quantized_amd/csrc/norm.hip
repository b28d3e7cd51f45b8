// The norms between two blocks, the residual between them and the quantiser
// behind them, in one pass over the row (gfx950).
//
//   n = y * rsqrt(mean(y^2) + eps) * post_weight       (n = y without one)
//   h = t(residual + residual_scale * (gate * n))      t: the 16-bit type
//   z = t(h * rsqrt(mean(h^2) + eps) * pre_weight)
//   q, s = the symmetric INT8 quantiser of z, per 1 x 128 group or per row
//
// Quantiser: the page "FP8 vs INT8 quantisation for DeepSeek", section 3.2.1
// (int8 branch), at the granularities of "DeepSeek R1 INT8 quantisation in
// SGLang", section 2.3.  The second norm reads h as it is stored (rounded to
// t) and the quantiser reads z rounded to t, so a layer that takes 16-bit
// inputs and one that takes the codes see the same activations, and the codes
// are those of quant_act_group / quant_act_token on z, bit for bit.  All else
// is fp32: squares, their sums, products.
#include "common.h"
#include "launch.h"

namespace w8 {
namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Sum or maximum over a workgroup of NW waves; every thread gets it.  red
// holds NW floats that nothing else uses between this call's barrier and the
// next call on the same array.
template <int NW>
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  if (NW == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float r = red[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) r += red[w];
  return r;
}

template <int NW>
__device__ __forceinline__ float block_max(float v, float* red) {
  v = wave_max(v);
  if (NW == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float r = red[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) r = fmaxf(r, red[w]);
  return r;
}

typedef float v2f __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));

// 8 fp32 values to the 16-bit type (round to nearest even), packed: one
// conversion instruction for two values.
template <bool FP16>
__device__ __forceinline__ uint4 pack8(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const v2f x = {v[2 * i], v[2 * i + 1]};
    if (FP16)
      w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, v2h));
    else
      w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, v2b));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One row of a 16-bit array (or an empty range where the array is absent) as
// a buffer: a load past its end, or of an absent array, reads zeros and moves
// nothing, so no load sits under a branch and all of a row's loads are under
// way before the first is waited for.
struct Row {
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ Row(const void* base, int64_t row, int K) {
    const uint64_t at = (uint64_t)base + (uint64_t)row * (uint64_t)K * 2;
    const uint64_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)at);
    const uint64_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(at >> 32));
    r = __builtin_amdgcn_make_buffer_rsrc((void*)(lo | (hi << 32)), 0, base ? K * 2 : 0, 0x00020000);
  }
  __device__ __forceinline__ uint4 chunk(int c) const {
    return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, c * 16, 0, 0));
  }
};

// One workgroup of NT threads per row; thread t holds the 8-value chunks t,
// t + NT, ... (CH of them at most), so the row is read once and stays in
// registers through both norms and the quantiser.  A 128-value group is the
// 16 chunks of 16 neighbouring lanes.  HBM-bound: 4096 x 7168 with residual,
// both norms and group codes 41 us, 206 MB at 5.0 TB/s; one row 4.4 us.
// (The same in 64-bit arithmetic throughout takes 58 and 6.4 us, and as much
// where only values near a border of the 16-bit type are done again in 64.)
// LATE: all but y is loaded where it is used instead, which leaves registers
// for two workgroups of 1024 threads per CU.
template <bool FP16, int NT, int CH, bool LATE>
__global__ __launch_bounds__(NT, LATE ? 8 : 1) void k_norm_residual_quant(NormArgs a) {
  constexpr int NW = NT / 64;
  __shared__ float red[3][NW];
  const int64_t row = a.row0 + blockIdx.x;
  const int nch = a.K >> 3;
  const Row y(a.y, row, a.K), res(a.residual, row, a.K), gate(a.gate, a.gate_rows == 1 ? 0 : row, a.K),
      pw(a.post_weight, 0, a.K), nw(a.pre_weight, 0, a.K);
  const float inv_k = 1.0f / (float)a.K;

  // whether this wave has any of the row's i-th chunks: in the wide shapes,
  // waves past the row's end skip the arithmetic (one row of 18432: 7.5 us
  // against 8.1; in the narrow ones the branches cost more than they save,
  // 4096 x 7168 41.6 us against 41.0)
  const int first = __builtin_amdgcn_readfirstlane((int)threadIdx.x & ~63);
  auto inside = [&](int i) { return NT * CH <= 1024 || first + NT * i < nch; };

  constexpr int CE = LATE ? 1 : CH;
  uint4 raw[CH], rr[CE], rg[CE], rp[CE], rn[CE];
#pragma unroll
  for (int i = 0; i < CH; ++i) raw[i] = y.chunk(threadIdx.x + NT * i);
#pragma unroll
  for (int i = 0; i < CE && !LATE; ++i) rr[i] = res.chunk(threadIdx.x + NT * i);
#pragma unroll
  for (int i = 0; i < CE && !LATE; ++i) {
    rg[i] = gate.chunk(threadIdx.x + NT * i);
    rp[i] = pw.chunk(threadIdx.x + NT * i);
    rn[i] = nw.chunk(threadIdx.x + NT * i);
  }
  float inv = 1.0f;
  if (a.post_weight) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (!inside(i)) break;
      float v[8];
      unpack8<FP16>(raw[i], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += v[e] * v[e];
    }
    inv = 1.0f / __builtin_sqrtf(block_sum<NW>(ss, red[0]) * inv_k + a.eps);
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    if (!inside(i)) break;
    const int c = threadIdx.x + NT * i;
    float v[8], o[8];
    unpack8<FP16>(raw[i], v);
    if (a.post_weight) {
      unpack8<FP16>(LATE ? pw.chunk(c) : rp[i % CE], o);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * inv * o[e];
    }
    if (a.gate) {
      unpack8<FP16>(LATE ? gate.chunk(c) : rg[i % CE], o);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= o[e];
    }
    unpack8<FP16>(LATE ? res.chunk(c) : rr[i % CE], o);   // zeros without a residual
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] * a.residual_scale + o[e];
    raw[i] = pack8<FP16>(v);
    if (c < nch) static_cast<uint4*>(a.h)[row * nch + c] = raw[i];
    unpack8<FP16>(raw[i], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += v[e] * v[e];
  }
  inv = 1.0f / __builtin_sqrtf(block_sum<NW>(ss, red[1]) * inv_k + a.eps);

  float am[CH];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    if (!inside(i)) break;
    const int c = threadIdx.x + NT * i;
    float v[8], o[8];
    unpack8<FP16>(raw[i], v);
    unpack8<FP16>(LATE ? nw.chunk(c) : rn[i % CE], o);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] * inv * o[e];
    raw[i] = pack8<FP16>(v);
    if (a.z && c < nch) static_cast<uint4*>(a.z)[row * nch + c] = raw[i];
    unpack8<FP16>(raw[i], v);
    am[i] = amax_n(v, 8);
    amax = fmaxf(amax, am[i]);
  }
  if (!a.q) return;
  const bool group = a.group;
  if (!group) amax = block_max<NW>(amax, red[2]);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    if (!inside(i)) break;
    const int c = threadIdx.x + NT * i;
    // a group's 16 lanes are all inside the row or all outside it
    const QScale sc = make_scale(group ? max16(am[i]) : amax);
    float v[8];
    unpack8<FP16>(raw[i], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = quant_one(v[e], sc);
    if (c < nch) {
      uint2 o;
      o.x = pack4(v[0], v[1], v[2], v[3]);
      o.y = pack4(v[4], v[5], v[6], v[7]);
      reinterpret_cast<uint2*>(a.q + row * (int64_t)a.K)[c] = o;
      if (group && (c & 15) == 0) a.q_scale[row * (a.K >> 7) + (c >> 4)] = sc.s;
    }
  }
  if (!group && threadIdx.x == 0) a.q_scale[row] = make_scale(amax).s;
}

// A launch holds fewer than 2^32 threads: rows in parts of 2^20.
template <bool FP16, int NT, int CH, bool LATE = false>
hipError_t norm_go(NormArgs a, int64_t M, hipStream_t st) {
  constexpr int64_t kPart = int64_t(1) << 20;
  for (a.row0 = 0; a.row0 < M; a.row0 += kPart) {
    const int64_t n = M - a.row0 < kPart ? M - a.row0 : kPart;
    hipLaunchKernelGGL((k_norm_residual_quant<FP16, NT, CH, LATE>), dim3((unsigned)n), dim3(NT), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Up to 256 rows, one to a CU, a row is spread over more threads; with more
// rows fewer and fuller threads win in the end.  Residual, both norms, group
// codes, us (threads x chunks):
//   K = 4096   64 rows 4.4 with 512 x 1, 5.1 with 256 x 2; 257 rows 5.0, 5.6;
//              333 rows 6.0, 6.1; 1023 rows 9.6, 9.4; 4096 rows 22.2, 20.3
//   K = 7168   64 rows 5.5 with 1024 x 1, 5.7 with 512 x 2; 257 rows 7.2, 6.9;
//              4096 rows 49, 41
//   K = 8320   64 rows 6.5 with 1024 x 2, 6.2 with 512 x 3; 257 rows 8.4, 8.2;
//              1023 rows 18.6, 16.3
//   K = 16384  64 rows 8.0 with 1024 x 2, 8.3 with 512 x 4; 1023 rows 24.6, 24.5
//   K = 18432  one row 7.4 with 1024 x 3, 7.8 with 1024 x 4; 1023 rows 37 with
//              every load first, 28 LATE
// So 256 is a little early at K = 4096 and late at 8320; either costs at most
// 0.6 us.  K <= 2048 has one shape: at 4096 rows of 512 three quarters of its
// threads idle (11 us; 1152 12.4 us, 2048 14.3 us).
template <bool FP16>
hipError_t norm_launch(const NormArgs& a, int64_t M, hipStream_t st) {
  const int nch = a.K >> 3;
  const bool few = M <= 256;
  if (nch <= 256) return norm_go<FP16, 256, 1>(a, M, st);
  if (nch <= 512) return few ? norm_go<FP16, 512, 1>(a, M, st) : norm_go<FP16, 256, 2>(a, M, st);
  if (nch <= 1024) return few ? norm_go<FP16, 1024, 1>(a, M, st) : norm_go<FP16, 512, 2>(a, M, st);
  if (few && nch <= 2048) return norm_go<FP16, 1024, 2>(a, M, st);
  if (few) return nch <= 3 * 1024 ? norm_go<FP16, 1024, 3>(a, M, st) : norm_go<FP16, 1024, 4>(a, M, st);
  if (nch <= 3 * 512) return norm_go<FP16, 512, 3>(a, M, st);
  if (nch <= 2048) return norm_go<FP16, 512, 4>(a, M, st);
  return nch <= 3 * 1024 ? norm_go<FP16, 1024, 3, true>(a, M, st) : norm_go<FP16, 1024, 4, true>(a, M, st);
}

}  // namespace

hipError_t launch_norm_residual_quant(const NormArgs& a, bool fp16, int64_t M, hipStream_t st) {
  return fp16 ? norm_launch<true>(a, M, st) : norm_launch<false>(a, M, st);
}

}  // namespace w8
