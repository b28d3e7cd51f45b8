// Keys and values quantised into the pages of a cache, and read back (gfx950).
//
//   s = fp32(max(amax, 1e-10) / 127 or / 7), q = clamp(rne(fp32(x / s)))
//
// per token and head: the symmetric quantiser of "FP8 vs INT8 quantisation for
// DeepSeek", section 3.2.1 (int8 branch), with a head's channels as its group.
// Layout of the pages: include/w8a8.h.
//
// Sixteen lanes hold a row (a sixteenth of the channels each, which is the unit
// in which values are stored) and a wave four tokens of one head, keys and
// values both, so the four fill a value block of their own with one store where
// their slots follow each other.  The four waves of a workgroup take
// neighbouring heads, workgroups neighbouring groups of heads, then the next
// four tokens: together they pass over contiguous memory.  All loads of a lane
// are issued before the first is used.  Bound by HBM in both directions for
// long calls and by the launch for a few tokens (128 channels, 4 bits, 8 heads):
// 65536 tokens are written in 75 us (340 MB, 4.5 TB/s), 32768 read back in 35 us
// with ten caches in turn (170 MB, 4.8 TB/s), where a large copy moves 4.9; one
// token takes 3.1 and 2.3 us.  Keys and values in workgroups of their own, a row
// after the other, took 98 us to write, and 33 to read two caches in turn (27.7
// now).  Heads that are no multiple of four leave waves idle: the same bytes as 8
// heads of 65536 tokens (84 us to write in one run of calls, 77 to read) took 77
// and 77 us as 4 heads, 80 and 82 as 3, 103 and 106 as 1, 105 and 107 as 5.  8 bits:
// 65536 tokens 82 us to write (5.0 TB/s), 76 to read back to 16 bits (5.3 TB/s).
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

// A lane's token, head and sixteenth; tokens to a workgroup: kTokens.
constexpr int kTokens = 4;
struct KvPlace {
  int64_t t;
  int h, c;
};
__device__ __forceinline__ KvPlace kv_place(const KvArgs& a) {
  const uint32_t groups = ((uint32_t)a.H + 3) / 4, at = blockIdx.x / groups;
  KvPlace p;
  p.t = (int64_t)at * kTokens + ((threadIdx.x >> 4) & 3);
  p.h = (int)((blockIdx.x - at * groups) * 4 + (threadIdx.x >> 6));
  p.c = threadIdx.x & 15;
  return p;
}

template <bool FP16, int D>
__device__ __forceinline__ void kv_unpack(const uint32_t* w, float* x) {
  constexpr int kC = D / 16;
  if constexpr (kC == 4) {
    float y[8];
    unpack8<FP16>(make_uint4(w[0], w[1], 0, 0), y);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = y[i];
  } else {
#pragma unroll
    for (int i = 0; i < kC / 8; ++i) unpack8<FP16>(make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]), x + 8 * i);
  }
}

// N * 4 bytes (8, 16 or 32).
template <int N>
__device__ __forceinline__ void get_words(const uint8_t* p, uint32_t* w) {
  if constexpr (N == 2) {
    get<8>(p, w);
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) get<16>(p + 16 * i, w + 4 * i);
  }
}
template <int N>
__device__ __forceinline__ void put_words(uint8_t* p, const uint32_t* w) {
  if constexpr (N == 2) {
    put<8>(p, w);
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) put<16>(p + 16 * i, w + 4 * i);
  }
}

// The codes of a lane's N values, packed: nibbles are joined as floats
// (q1 16 + q0 + 136, exact) and converted into their byte.  (One branch for all
// values that lie near a half-integer, instead of one for each, is slower:
// among 16-bit values half the largest one is common, which 4 bits put at 3.5.)
template <int N, int BITS>
__device__ __forceinline__ void kv_codes(const float* x, QScale s, uint32_t* w) {
  float t[N];
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = quant_one(x[i], s);
  if constexpr (BITS == 4) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      w[i / 4] = __builtin_amdgcn_cvt_pk_u8_f32(__builtin_fmaf(t[2 * i + 1], 16.f, t[2 * i] + 136.f), i & 3,
                                                i & 3 ? w[i / 4] : 0u);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      w[i / 4] = __builtin_amdgcn_cvt_pk_u8_f32(t[i] + 128.f, i & 3, i & 3 ? w[i / 4] : 0u);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) w[i] ^= 0x80808080u;   // offset to two's complement
  }
}

template <bool FP16, int D, int BITS>
__global__ __launch_bounds__(256) void k_kv_write(KvArgs a) {
  constexpr int kC = D / 16, kDB = D * BITS / 8, kN = kDB / 16;   // channels and bytes to a lane
  const KvPlace p = kv_place(a);
  if (p.h >= a.H || p.t >= a.T) return;
  const int32_t slot = a.slots[p.t];
  const int64_t at = (int64_t)p.h * D + p.c * kC;
  uint32_t w16[2][kC / 2];
  get_words<kC / 2>(reinterpret_cast<const uint8_t*>(static_cast<const uint16_t*>(a.k16) + p.t * a.k_stride + at), w16[0]);
  get_words<kC / 2>(reinterpret_cast<const uint8_t*>(static_cast<const uint16_t*>(a.v16) + p.t * a.v_stride + at), w16[1]);
  if (slot < 0 || slot >= a.slots_end) return;   // (whole rows: sixteen lanes)
  const int page = slot / a.page, off = slot - page * a.page;
  const int64_t row0 = ((int64_t)page * a.H + p.h) * a.page;
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    float x[kC];
    kv_unpack<FP16, D>(w16[v], x);
    const float amax = max16(amax_n(x, kC));
    const QScale s = BITS == 4 ? make_scale4(amax) : make_scale(amax);
    uint32_t w[4] = {0, 0, 0, 0};
    kv_codes<kC, BITS>(x, s, w);
    put<kN>((v ? a.v : a.k) + code_at<kDB>(v != 0, row0, off, p.c), w);
    if (p.c == 0) (v ? a.vs : a.ks)[row0 + off] = s.s;
  }
}

// The same rows back: code times scale in fp32, rounded once.  OUT: a w8_dtype.
template <int OUT, int D, int BITS>
__global__ __launch_bounds__(256) void k_kv_read(KvArgs a) {
  constexpr int kC = D / 16, kDB = D * BITS / 8, kN = kDB / 16;
  const KvPlace p = kv_place(a);
  if (p.h >= a.H || p.t >= a.T) return;
  const int32_t slot = a.slots[p.t];
  uint32_t w[2][4] = {};
  float s[2] = {0.f, 0.f};
  const bool there = slot >= 0 && slot < a.slots_end;
  if (there) {
    const int page = slot / a.page, off = slot - page * a.page;
    const int64_t row0 = ((int64_t)page * a.H + p.h) * a.page;
    get<kN>(a.k + code_at<kDB>(false, row0, off, p.c), w[0]);
    get<kN>(a.v + code_at<kDB>(true, row0, off, p.c), w[1]);
    s[0] = a.ks[row0 + off];
    s[1] = a.vs[row0 + off];
  }
  const int64_t at = (p.t * a.H + p.h) * D + p.c * kC;
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    float x[kC];
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      if constexpr (BITS == 4) x[i] = (float)((int)((w[v][i / 8] >> (4 * (i & 7))) & 15u) - 8) * s[v];
      else x[i] = (float)(int)(int8_t)(w[v][i / 4] >> (8 * (i & 3))) * s[v];
      if (!there) x[i] = 0.f;
    }
    uint8_t* const out = static_cast<uint8_t*>(v ? a.v_out : a.k_out) + at * (OUT == 2 ? 4 : 2);
    if constexpr (OUT == 2) {
#pragma unroll
      for (int i = 0; i < kC / 4; ++i)
        *reinterpret_cast<v4f*>(out + 16 * i) = v4f{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
    } else {
      uint32_t o[kC / 2];
#pragma unroll
      for (int i = 0; i < kC / 2; ++i) {
        const v2f y = {x[2 * i], x[2 * i + 1]};
        if constexpr (OUT == 1) o[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, v2h));
        else o[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, v2b));
      }
      put_words<kC / 2>(out, o);
    }
  }
}

template <int D, int BITS>
hipError_t kv_go(const KvArgs& a, bool write, int dtype, hipStream_t st) {
  const int64_t blocks = (a.T + kTokens - 1) / kTokens * ((a.H + 3) / 4);
  const dim3 grid((unsigned)blocks), wg(256);
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

hipError_t launch_kv(const KvArgs& a, bool write, int dtype, int bits, int D, hipStream_t st) {
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
