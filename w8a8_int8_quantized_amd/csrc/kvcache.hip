// Keys and values quantised into the pages of a cache, and read back (gfx950).
//
//   s = fp32(max(amax, 1e-10) / 127 or / 7), q = clamp(rne(fp32(x / s)))
//
// per token and head: the symmetric quantiser of "FP8 vs INT8 quantisation for
// DeepSeek", section 3.2.1 (int8 branch), with a head's channels as its group.
// Layout of the pages: include/w8a8.h.
//
// Sixteen lanes hold a row (a sixteenth of the channels each, which is the unit
// in which values are stored), so the four tokens that a wave takes of one head
// fill a value block of their own with one store where their slots follow each
// other.  Bound by HBM for prompts and by the launch for a few tokens.
#include "common.h"
#include "launch.h"

namespace w8 {
namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));

// N bytes (2, 4, 8 or 16) between registers and an N-byte aligned address.
template <int N>
__device__ __forceinline__ void put(uint8_t* p, const uint32_t* w) {
  if constexpr (N == 2) *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
  else if constexpr (N == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
  else if constexpr (N == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <int N>
__device__ __forceinline__ void get(const uint8_t* p, uint32_t* w) {
  if constexpr (N == 2) {
    w[0] = *reinterpret_cast<const uint16_t*>(p);
  } else if constexpr (N == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  }
}

// Byte address of sixteenth c of a token's key, or of its value, in a cache
// whose rows hold DB bytes: row0 counts tokens [pages][Hkv][page] up to the
// page's and head's first, off is the token's place in the page.
template <int DB>
__device__ __forceinline__ int64_t code_at(bool value, int64_t row0, int off, int c) {
  if (!value) return (row0 + off) * DB + c * (DB / 16);
  return row0 * DB + (int64_t)(off >> 2) * (4 * DB) + c * (DB / 4) + (off & 3) * (DB / 16);
}

// One row to sixteen lanes: rows are token x head, tokens fastest, so that the
// four rows of a wave are four tokens of a head.  blockIdx.y: keys, values.
template <bool FP16, int D, int BITS>
__global__ __launch_bounds__(256) void k_kv_write(KvArgs a) {
  constexpr int kC = D / 16, kDB = D * BITS / 8, kN = kDB / 16;   // channels and bytes to a lane
  const bool value = blockIdx.y != 0;
  const int c = threadIdx.x & 15;
  const int64_t row = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int64_t h = row / a.T4, t = row - h * a.T4;   // T4: T rounded up to a multiple of 4
  if (h >= a.H || t >= a.T) return;
  const int32_t slot = a.slots[t];
  if (slot < 0 || slot >= a.slots_end) return;
  const uint16_t* src = static_cast<const uint16_t*>(value ? a.v16 : a.k16) + t * (value ? a.v_stride : a.k_stride) +
                        h * D + c * kC;
  float x[kC];
  if constexpr (kC == 4) {
    const uint2 w = *reinterpret_cast<const uint2*>(src);
    float y[8];
    unpack8<FP16>(make_uint4(w.x, w.y, 0, 0), y);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = y[i];
  } else {
#pragma unroll
    for (int i = 0; i < kC / 8; ++i) unpack8<FP16>(*reinterpret_cast<const uint4*>(src + 8 * i), x + 8 * i);
  }
  const float amax = max16(amax_n(x, kC));
  const QScale s = BITS == 4 ? make_scale4(amax) : make_scale(amax);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    const int q = (int)quant_one(x[i], s);
    if constexpr (BITS == 4) w[i / 8] |= (uint32_t)(q + 8) << (4 * (i & 7));
    else w[i / 4] |= ((uint32_t)q & 0xffu) << (8 * (i & 3));
  }
  const int page = slot / a.page, off = slot - page * a.page;
  const int64_t row0 = ((int64_t)page * a.H + h) * a.page;
  put<kN>((value ? a.v : a.k) + code_at<kDB>(value, row0, off, c), w);
  if (c == 0) (value ? a.vs : a.ks)[row0 + off] = s.s;
}

// The same rows back: code times scale in fp32, rounded once.  OUT: a w8_dtype.
template <int OUT, int D, int BITS>
__global__ __launch_bounds__(256) void k_kv_read(KvArgs a) {
  constexpr int kC = D / 16, kDB = D * BITS / 8, kN = kDB / 16;
  const bool value = blockIdx.y != 0;
  const int c = threadIdx.x & 15;
  const int64_t row = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int64_t h = row / a.T4, t = row - h * a.T4;
  if (h >= a.H || t >= a.T) return;
  const int32_t slot = a.slots[t];
  float x[kC];
#pragma unroll
  for (int i = 0; i < kC; ++i) x[i] = 0.f;
  if (slot >= 0 && slot < a.slots_end) {
    const int page = slot / a.page, off = slot - page * a.page;
    const int64_t row0 = ((int64_t)page * a.H + h) * a.page;
    uint32_t w[4];
    get<kN>((value ? a.v : a.k) + code_at<kDB>(value, row0, off, c), w);
    const float s = (value ? a.vs : a.ks)[row0 + off];
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      if constexpr (BITS == 4) x[i] = (float)((int)((w[i / 8] >> (4 * (i & 7))) & 15u) - 8) * s;
      else x[i] = (float)(int)(int8_t)(w[i / 4] >> (8 * (i & 3))) * s;
    }
  }
  const int64_t at = (t * a.H + h) * D + c * kC;
  if constexpr (OUT == 2) {
    float* out = static_cast<float*>(value ? a.v_out : a.k_out) + at;
#pragma unroll
    for (int i = 0; i < kC / 4; ++i)
      *reinterpret_cast<v4f*>(out + 4 * i) = v4f{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
  } else {
    uint32_t w[kC / 2];
#pragma unroll
    for (int i = 0; i < kC / 2; ++i) {
      const v2f p = {x[2 * i], x[2 * i + 1]};
      if constexpr (OUT == 1) w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, v2h));
      else w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, v2b));
    }
    uint8_t* out = static_cast<uint8_t*>(value ? a.v_out : a.k_out) + at * 2;
    if constexpr (kC == 4) put<8>(out, w);
    else {
#pragma unroll
      for (int i = 0; i < kC / 8; ++i) put<16>(out + 16 * i, w + 4 * i);
    }
  }
}

template <int D, int BITS>
hipError_t kv_go(const KvArgs& a, bool write, int dtype, hipStream_t st) {
  const int64_t blocks = (a.T4 * a.H + 15) / 16;
  const dim3 grid((unsigned)blocks, 2), wg(256);
  if (write) {
    if (dtype == 1) hipLaunchKernelGGL((k_kv_write<true, D, BITS>), grid, wg, 0, st, a);
    else hipLaunchKernelGGL((k_kv_write<false, D, BITS>), grid, wg, 0, st, a);
  } else {
    if (dtype == 0) hipLaunchKernelGGL((k_kv_read<0, D, BITS>), grid, wg, 0, st, a);
    else if (dtype == 1) hipLaunchKernelGGL((k_kv_read<1, D, BITS>), grid, wg, 0, st, a);
    else hipLaunchKernelGGL((k_kv_read<2, D, BITS>), grid, wg, 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv(KvArgs a, bool write, int dtype, int bits, int D, hipStream_t st) {
  a.T4 = (a.T + 3) & ~int64_t(3);
  if (bits == 4) {
    if (D == 64) return kv_go<64, 4>(a, write, dtype, st);
    if (D == 128) return kv_go<128, 4>(a, write, dtype, st);
    return kv_go<256, 4>(a, write, dtype, st);
  }
  if (D == 64) return kv_go<64, 8>(a, write, dtype, st);
  if (D == 128) return kv_go<128, 8>(a, write, dtype, st);
  return kv_go<256, 8>(a, write, dtype, st);
}

}  // namespace w8
