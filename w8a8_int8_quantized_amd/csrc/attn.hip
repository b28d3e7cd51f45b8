// Attention over a key/value cache held in 4 or 8 bits (gfx950).
//
//   s[t] = scale * ks[t] * sum_d q[d] kc[t][d]        kc, vc: integer codes
//   p[t] = exp(s[t] - m),  l = sum_t p[t]
//   o[d] = (sum_t p[t] vs[t] vc[t][d]) / l,  lse = m + ln l
//
// The codes are those of the symmetric quantiser of "FP8 vs INT8 quantisation
// for DeepSeek", section 3.2.1 (int8 branch), with one scale per token and
// head, so a scale is one factor of a column of s or p and the matrix
// instructions see integers, which 16-bit floats hold exactly.
//
// Layout of the work.  S^T = K Q^T and O^T = V^T P^T by 16x16x32 matrix
// instructions: a lane's column is a query row in both, and the four tokens of
// each half tile that it holds of S^T are the tokens that it feeds into P^T,
// so probabilities never leave the lane.  Keys lie by token: a lane reads a
// quarter of a token's channels.  Values lie in blocks of four tokens by
// sixteenths of the channels (include/w8a8.h): a lane reads its four tokens'
// sixteenth, and bytes of two tokens are joined by one byte permutation.
//
// Each wave streams its tiles through a ring of its own in LDS, filled by
// direct-to-LDS loads that read memory in order: no registers and no barriers.
// Keys are swizzled within a row on the way, so that the fragment reads meet no
// bank conflicts.  One tile is in flight while the one before it is computed up
// to its probabilities, whatever the ring's depth: the compiler waits for all
// loads in front of the two page ids of the next tile, as the register that
// holds them is loaded in a branch (`next` below).
//
// Codes to 16-bit floats: OR an exponent on top of the code bits in place,
// which gives 2^k + code + offset exactly.  For the keys the constant is not
// subtracted from each but once from the sum: the accumulators start at
// -(2^k + offset) * sum_d q[d].  For the values it is subtracted (exact in
// fp16): a running sum over a long cache must not carry an offset that is
// larger than its result.  The sum of a score does carry it: scores of ordinary
// queries (around 0) are off by 1e-6 to 3e-5 for it, those of fp16 queries of
// mean 8, with 256 channels of 4 bits, by up to 1.2e-3 (a subtraction per pair of
// codes is 32 vector instructions a tile for it, and bf16 has no packed one).
//
// Softmax: a row's probabilities are exp2(s - m) with a reference m that the
// largest term p vs passes by 2^10 to 2^15 before it moves (one compare a
// tile), so the accumulators are seldom rescaled.  p vs goes into the second
// product as fp16: half a step is 2^-11 of the term, and what lies 2^-24 below
// the largest is rounded to that.  References, l and all sums are fp32; the
// reference cancels in o = O / l.  Where scores pass 2^20 a step of fp32 is too
// coarse for a reference that also holds the 2^10 and the scale: such rows take
// a way of their own (rare_references), as do value scales that are not finite.
// Ordinary rows pay for it with a scalar test a tile and compares where
// references move and in masked tiles (0 to 2 % of a call, 2 to 4 % with 8 bits
// in 64 rows).
//
// Work is shared out in equal runs of 32-token tiles over all sequences and
// heads (attn_plan.h); the waves of a workgroup take parts of a segment's run
// and join in LDS; a segment that more than one workgroup holds is joined by
// a second kernel, in order, so results do not depend on timing.  Short
// segments have a workgroup of up to 16 waves each, and no second kernel.
//
// What bounds it.  Decoding: reads with one tile of each wave in flight.  64
// sequences of 1 to 16384 tokens (32 query heads on 8, 128 channels, 4 bits, 473
// MB) take 97 us, 4.9 TB/s, where pure reads reach 6.3; of 98.9 us, the loads
// without the computation took 94.6, with that wait in them, and the computation
// without the loads 66.5.  Tiles in registers instead of the LDS ring took 134 us
// (the kernel alone, 94 now; other steps lie between).  Prompts: the vector pipe,
// which takes the codes apart and does the softmax (by counters, 472 vector
// instructions for 64 matrix ones, 64 rows of 32 tokens): 2048 tokens on 8192
// take 311 us, 780 TFLOP/s, where a large bf16 library product does 1219.  With 128
// channels of 4 bits in 64 rows 39 vector registers do not fit and lie in scratch
// (36 with fp16), some of them read back in the tile loop; 52 of the 140 kernels
// keep scalars in vector lanes.  Few tokens: a chain of loads (lengths, page ids
// and queries, tiles) and, where segments are shared, the second kernel (5 to 7
// us traced).
#include "attn_plan.h"
#include "common.h"
#include "launch.h"
#include "pipeline.h"

namespace w8 {
namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

constexpr float kUnset = -3.4028235e38f;  // a reference before the first score: the least number
constexpr float kFar = 1048576.f;         // 2^20: references from here on keep their lift apart
constexpr float kLift = 10.f;             // log2 of what the largest p vs becomes
constexpr float kTermLimit = 32768.f;     // what p vs may grow to: fp16 ends at 65504
constexpr float kSumLimit = 1.2676506e30f;   // what a sum of p may grow to within a tile, 2^100
constexpr float kTinyScale = 5.9604645e-8f;  // 2^-24: a value scale counts as this at least in the reference
constexpr float kLn2 = 0.693147180559945309f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// ln(l 2^m): the exponents are added exactly before the logarithm's rounding.
__device__ __forceinline__ float log_sum(float m, float l) {
  const float e = (float)__builtin_amdgcn_frexp_expf(l);
  return l == 0.f ? -__builtin_inff() : kLn2 * ((m + e) + __log2f(__builtin_amdgcn_frexp_mantf(l)));
}

// Across the lanes of a row: lane ^ FROM, lane ^ 2 FROM, .. lane ^ 32.
template <int FROM>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int d = FROM; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}
template <int FROM>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int d = FROM; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// `to`, with the lanes of bank B (4 B .. 4 B + 3 of each 16) taken from x, SH
// lanes below.
template <int SH, int BANKS>
__device__ __forceinline__ float from_below(float to, float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(to), __float_as_int(x), 0x110 + SH, 0xF, BANKS, false));
}
// x of the lane SH above within the 16 (0 past the end).
template <int SH>
__device__ __forceinline__ uint32_t from_above(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x100 + SH, 0xF, 0xF, true);
}

// 16 bytes per lane from base + voff into LDS at lds + 16 lane, and 4 bytes per
// lane from an address of its own into lds + 4 lane.  No register result, so
// nothing can be overwritten while a load is in flight; the caller counts them.
// (The wait states: M0 and the base may have been written just before.)
__device__ __forceinline__ void dma_rows(const uint8_t* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
               ::"s"(lds), "v"(voff), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void dma_rows_at(const uint8_t* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, off"
               ::"s"(lds), "v"(p) : "memory", "m0");
}
__device__ __forceinline__ void dma_word_at(const uint8_t* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, off"
               ::"s"(lds), "v"(p) : "memory", "m0");
}
// All but N of the wave's vector memory operations are done.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// ------------------------------------------------------------ codes to floats
// (x & mask) | exponent in one instruction: one operand of v_and_or_b32 can be
// a constant, so the exponents stay in registers that the compiler is kept from
// seeing through.
__device__ __forceinline__ uint32_t held(uint32_t c) {
  asm("" : "+v"(c));
  return c;
}
struct Exponents {
  uint32_t key, lo, hi;           // of the key codes, and of the low and high nibbles (or bytes) of values
};

// The key operand of one matrix instruction, 8 channels of a lane's quarter.
// 4 bits: channels in the order 0 4 1 5 2 6 3 7 (the query's operand has the
// same), value 128 + n (bf16) or 64 + n (fp16), n = code + 8.  8 bits: in
// order, value code + 128 (bf16) or 1024 + code + 128 (fp16).
template <bool FP16, int BITS>
struct KeyCodes {
  static constexpr float kOffset = BITS == 4 ? (FP16 ? 72.f : 136.f) : (FP16 ? 1152.f : 128.f);
  static constexpr uint32_t kExp = BITS == 4 ? (FP16 ? 0x54005400u : 0x43004300u) : 0x64646464u;
  static __device__ __forceinline__ v4u operand(const uint32_t* w, uint32_t e) {
    v4u r;
    if constexpr (BITS == 4 && FP16) {
      r[0] = ((w[0] << 4) & 0x00F000F0u) | e;
      r[1] = (w[0] & 0x00F000F0u) | e;
      r[2] = ((w[0] >> 4) & 0x00F000F0u) | e;
      r[3] = ((w[0] >> 8) & 0x00F000F0u) | e;
    } else if constexpr (BITS == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = ((w[0] >> (4 * i)) & 0x000F000Fu) | e;
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t u = w[i] ^ 0x80808080u;
        if constexpr (FP16) {
          r[2 * i] = __builtin_amdgcn_perm(e, u, 0x04010400u);
          r[2 * i + 1] = __builtin_amdgcn_perm(e, u, 0x04030402u);
        } else {
          const uint32_t f0 = __float_as_uint((float)(u & 0xffu)), f1 = __float_as_uint((float)((u >> 8) & 0xffu));
          const uint32_t f2 = __float_as_uint((float)((u >> 16) & 0xffu)), f3 = __float_as_uint((float)(u >> 24));
          r[2 * i] = __builtin_amdgcn_perm(f1, f0, 0x07060302u);       // integers below 256: the low halves are 0
          r[2 * i + 1] = __builtin_amdgcn_perm(f3, f2, 0x07060302u);
        }
      }
    }
    return r;
  }
};

// Byte B of two tokens T, T + 1 of a value unit (four tokens of DV bytes): in
// the low bytes of the two halves.
template <int DV, int T, int B>
__device__ __forceinline__ uint32_t token_pair(const uint32_t* w) {
  constexpr int o0 = T * DV + B, o1 = (T + 1) * DV + B;
  constexpr uint32_t sel = 0x0c000c00u | (uint32_t)(o0 & 3) | ((uint32_t)(4 + (o1 & 3)) << 16);
  return __builtin_amdgcn_perm(w[o1 >> 2], w[o0 >> 2], sel);
}

__device__ __forceinline__ uint32_t less(uint32_t h, float by) {
  const v2h b = {(_Float16)by, (_Float16)by};
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, h) - b);
}

// --------------------------------------------------------------- one segment
template <bool FP16, int D, int BITS, int ROWS, bool WHOLE>
struct Attn {
  static constexpr int R = ROWS > 16 ? ROWS / 16 : 1;      // row fragments of 16 columns
  // Up to 4 or 8 rows leave most of a fragment's columns empty.  The scores of
  // a lane's 8 tokens then move to PK lanes of its 16 (2 or 4 to each), where
  // exp and the rest of the softmax run without empty lanes, and back as
  // packed fp16.
  static constexpr int PK = ROWS < 16 ? 16 / ROWS : 1;
  static constexpr int kPer = 8 / PK;                     // scores of a lane and fragment in the softmax
  static constexpr int kDB = D * BITS / 8;          // bytes of a token's codes
  static constexpr int kW = kDB / 16;               // dwords of a lane per half tile, keys or values
  static constexpr int kSteps = D / 32;             // matrix instructions per half tile of S^T
  static constexpr int kJ = D / 16;                 // channels of a sixteenth: accumulators of O^T
  static constexpr int kRows = ROWS;
  static constexpr int kRound = 8;                  // accumulators (of 4) per round through LDS
  // With more than one row fragment the query operand and the accumulators'
  // starting values lie in LDS, one copy to the workgroup: the registers hold
  // the accumulators of up to 64 rows of 128 channels instead.
  static constexpr bool kQueryLds = R > 1;
  static constexpr int kQueryBytes = kQueryLds ? R * (kSteps + 1) * 1024 : 0;
  using KC = KeyCodes<FP16, BITS>;

  // A tile in LDS: the half tiles' keys and values (16 tokens each), 4 x 16 kDB
  // bytes, then 32 key and 32 value scales.
  static constexpr int kHalf = 16 * kDB;
  static constexpr int kTileBytes = 4 * kHalf + 256;
  static constexpr int kLoads = 4 * kHalf / 1024 + 1;    // loads to a tile
  // Tiles in a wave's ring.  (Three of 4 KB: 107 us where two took 105, with the
  // wait in front of page ids in both, and 16 waves of three do not fit in LDS.)
  static constexpr int kDepth = kDB == 32 ? 4 : 2;
  static constexpr int kRingBytes = kDepth * kTileBytes;
  // Waves to a workgroup; one that takes whole segments (short ones) has as
  // many as LDS holds rings for.
  static constexpr int kWaves = WHOLE ? attn_whole_waves(kDB) : kAttnWaves;
  static constexpr int kJoinBytes = kWaves * kRound * 4 * 64 * 4;
  static constexpr int kLdsBytes = kWaves * kRingBytes > kJoinBytes ? kWaves * kRingBytes : kJoinBytes;

  struct State {
    v4f o[R][kJ];
    float m[R], l[R];
    bool far;       // (of the wave) a row's reference passes kFar
  };

  static __device__ __forceinline__ v4f mma(const v4u& a, const v4u& b, const v4f& c) {
    if constexpr (FP16)
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0,
                                                     0);
  }
  static __device__ __forceinline__ v4f mma_h(const v4u& a, const v4u& b, const v4f& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  }

  // Where the lane's 16 bytes of a load lie in the 1024 that it moves, keys and
  // values (kDB = 32: in the 512 of its half tile).  Keys: chunk c of row m is
  // stored at c ^ key_swizzle(m), values with four chunks to a unit at
  // i ^ (unit / 4).
  static __device__ __forceinline__ uint32_t key_swizzle(uint32_t m) {
    if constexpr (kDB == 32) return (m >> 3) & 1;
    else if constexpr (kDB == 64) return (m >> 2) & 3;
    else if constexpr (kDB == 128) return m & 7;
    else return m & 15;
  }
  static __device__ __forceinline__ uint32_t value_swizzle(uint32_t unit) {
    return kDB == 256 ? (unit >> 2) & 3 : 0;
  }

  struct Lane {
    uint32_t k[4], v;           // offsets of the lane's bytes in global memory; k: per load of a half tile (kDB = 256)
    const uint8_t* scales;      // its scale at row 0
    uint32_t lk, lv, ls;        // offsets of its keys, values and scales in a tile in LDS
    int tok;                    // the first token whose probability it computes
    int lane;
  };
  static __device__ __forceinline__ Lane lane_of(const AttnArgs& a, int lane) {
    Lane l;
    const uint32_t m = lane & 15, g = lane >> 4;
    constexpr uint32_t kChunks = kDB / 16;              // 16-byte chunks of a row
    const uint32_t at = kDB == 32 ? lane & 31 : lane;   // position in the load, in chunks
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      const uint32_t row = (at + 64 * i) / kChunks, c = at % kChunks;
      l.k[i] = row * kDB + ((c ^ key_swizzle(row)) << 4);
    }
    // (a load of 64 chunks is 16 units of 4: the same pattern in each load)
    l.v = kDB == 256 ? (at & ~3u) * 16 + (((at & 3) ^ value_swizzle(at >> 2)) << 4) : at * 16;
    l.scales = reinterpret_cast<const uint8_t*>((lane < 32 ? a.ks : a.vs) + m);
    l.lk = m * kDB;
    l.lv = 2 * kHalf + (g * 16 + m) * (kDB / 4);
    const uint32_t v0 = PK == 1 ? 0 : (m / ROWS) * kPer;   // the lane's first score of its row's eight
    l.tok = 16 * (v0 >> 2) + 4 * g + (v0 & 3);
    l.ls = 4 * kHalf + l.tok * 4;
    l.lane = lane;
    return l;
  }

  // base0, base1: the half tiles' first token as a row of [pages][Hkv][page].
  static __device__ __forceinline__ void load(const AttnArgs& a, const Lane& l, int64_t base0, int64_t base1, uint32_t lds) {
    if constexpr (kDB == 32) {
      const int64_t row = l.lane & 32 ? base1 : base0;
      dma_rows_at(a.k + row * kDB + l.k[0], lds);
      dma_rows_at(a.v + row * kDB + l.v, lds + 1024);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < kHalf / 1024; ++i) dma_rows(a.k + (h ? base1 : base0) * kDB, l.k[i], lds + h * kHalf + i * 1024);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < kHalf / 1024; ++i)
          dma_rows(a.v + (h ? base1 : base0) * kDB + i * 1024, l.v, lds + (2 + h) * kHalf + i * 1024);
    }
    dma_word_at(l.scales + 4 * (l.lane & 16 ? base1 : base0), lds + 4 * kHalf);
  }

  // Half h of a tile in LDS: the lane's keys, values, and scales.
  static __device__ __forceinline__ void keys(const uint8_t* tile, const Lane& l, int h, uint32_t* w) {
    const uint32_t m = l.lane & 15, g = l.lane >> 4;
    if constexpr (kDB == 32) {
      const uint2 v = *reinterpret_cast<const uint2*>(tile + h * kHalf + l.lk + (((g >> 1) ^ key_swizzle(m)) << 4) +
                                                      (g & 1) * 8);
      w[0] = v.x;
      w[1] = v.y;
    } else {
#pragma unroll
      for (uint32_t i = 0; i < kDB / 64; ++i) {
        const uint32_t c = (g * (kDB / 64) + i) ^ key_swizzle(m);
        const v4u v = *reinterpret_cast<const v4u*>(tile + h * kHalf + l.lk + (c << 4));
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
      }
    }
  }
  static __device__ __forceinline__ void values_of(const uint8_t* tile, const Lane& l, int h, uint32_t* w) {
    if constexpr (kDB == 32) {
      const uint2 v = *reinterpret_cast<const uint2*>(tile + h * kHalf + l.lv);
      w[0] = v.x;
      w[1] = v.y;
    } else {
#pragma unroll
      for (uint32_t i = 0; i < kDB / 64; ++i) {
        const uint32_t c = i ^ value_swizzle(l.lane);
        const v4u v = *reinterpret_cast<const v4u*>(tile + h * kHalf + l.lv + (c << 4));
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
      }
    }
  }

  // The scores of a tile in codes.  qf: the query operand in registers, or in
  // LDS (ql, at the lane's place).
  static __device__ __forceinline__ void scores(const uint8_t* tile, const Lane& l, const v4u (*qf)[kSteps],
                                                const uint8_t* ql, const float* c0, const Exponents& e, v4f (*s)[2]) {
    if constexpr (kQueryLds) {
      uint32_t w[2][kW];
      keys(tile, l, 0, w[0]);
      keys(tile, l, 1, w[1]);
#pragma unroll
      for (int r = 0; r < R; ++r) s[r][0] = s[r][1] = *reinterpret_cast<const v4f*>(ql + (R * kSteps + r) * 1024);
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        // all fragments' operands are on their way before the codes are taken apart
        v4u q[R];
#pragma unroll
        for (int r = 0; r < R; ++r) q[r] = *reinterpret_cast<const v4u*>(ql + (r * kSteps + j) * 1024);
        __builtin_amdgcn_sched_barrier(0);
        const v4u k0 = KC::operand(w[0] + j * (BITS / 4), e.key), k1 = KC::operand(w[1] + j * (BITS / 4), e.key);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          s[r][0] = mma(k0, q[r], s[r][0]);
          s[r][1] = mma(k1, q[r], s[r][1]);
        }
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[kW];
        keys(tile, l, h, w);
        s[0][h] = v4f{c0[0], c0[0], c0[0], c0[0]};
#pragma unroll
        for (int j = 0; j < kSteps; ++j) s[0][h] = mma(KC::operand(w + j * (BITS / 4), e.key), qf[0][j], s[0][h]);
      }
    }
  }

  // Row r's sums in units of another reference, m.
  static __device__ __forceinline__ void move(int r, float m, float by, State& st) {
    st.m[r] = m;
    st.l[r] *= by;
#pragma unroll
    for (int j = 0; j < kJ; ++j) st.o[r][j] *= by;
  }

  // The references of a tile with far scores, or with value scales that are not
  // finite.  m: the new references, by: what takes the sums to them; s f - ref
  // become the exponents.
  //
  // At a far score a step of fp32 is more than the powers of two that p vs has
  // room for, and the fused product that an exponent begins with lies up to half
  // a step beside its rounding.  So the products are rounded first, the reference
  // is the largest score itself, and its lift (what takes the largest term to
  // kLift) is kept apart, in LDS, and added to the difference.  A wave that has
  // such a row comes here with all its tiles.
  //
  // A scale that is not finite must not reach rows that do not see its token,
  // and 0 times it would.  It becomes 0, and the rows that see it get NaN.
  static __device__ __forceinline__ void rare_references(float (*s)[kPer], float* f, float* vs, float* lifts, float* m,
                                                         float* by, float* ref, State& st) {
    int at = (int)threadIdx.x & (ROWS < 16 ? ROWS - 1 : 15);
    asm volatile("" : "+v"(at));   // (computed here, not held through the loop over the tiles)
    bool far = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float top = -__builtin_inff(), e = -__builtin_inff(), sees = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        s[r][i] *= f[i];
        top = fmaxf(top, s[r][i]);
        if (!(__builtin_fabsf(vs[i]) < __builtin_inff()) && s[r][i] != -__builtin_inff()) sees = 1.f;
      }
      top = row_max<16 / PK>(top);
      sees = row_max<16 / PK>(sees);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float v = __builtin_fabsf(vs[i]) < __builtin_inff() ? fmaxf(vs[i], kTinyScale) : kTinyScale;
        e = fmaxf(e, (s[r][i] - top) + __log2f(v));
      }
      const float to = kLift - row_max<16 / PK>(e), was = st.far ? lifts[16 * r + at] : 0.f;
      // up from m - was to top - to (and to an infinite top, where the difference is NaN)
      const bool up = !((top - st.m[r]) + (was - to) <= 0.f), apart = __builtin_fabsf(top) >= kFar;
      const float lift = up ? (apart ? to : 0.f) : was;
      m[r] = up ? (apart ? top : top - to) : st.m[r];
      by[r] = up ? exp2_hw((st.m[r] - m[r]) + (lift - was)) : 1.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) s[r][i] = (s[r][i] - m[r]) + lift;
      ref[r] = 0.f;
      far |= up && apart;
      lifts[16 * r + at] = lift;
      const float spoil = sees != 0.f ? __builtin_nanf("") : 1.f;
#pragma unroll
      for (int j = 0; j < kJ; ++j) st.o[r][j] *= spoil;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      f[i] = 1.f;
      vs[i] = __builtin_fabsf(vs[i]) < __builtin_inff() ? vs[i] : 0.f;
    }
    st.far |= __builtin_amdgcn_readfirstlane((int)(__ballot(far) != 0)) != 0;
  }

  // The probabilities of tokens t0 .. t0 + 31 of the sequence, times the value
  // scales, as fp16.  seen: the keys that the lane's rows see; all: whether
  // every row sees the whole tile.  lifts: of the wave's rows, in LDS.
  static __device__ __forceinline__ void softmax(const uint8_t* tile, const Lane& l, const v4f (*sc)[2],
                                                 float scale_log2, int t0, bool all, int L, const int* seen,
                                                 float* lifts, State& st, v4u* pf) {
    // score i of the lane: token l.tok + (i & 3) of half tile i / 4
    float s[R][kPer], f[kPer], vs[kPer];
    if constexpr (kPer == 2) {
      const v2f k = *reinterpret_cast<const v2f*>(tile + l.ls), v = *reinterpret_cast<const v2f*>(tile + l.ls + 128);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[i] = k[i] * scale_log2;
        vs[i] = v[i];
        s[0][i] = from_below<4, 2>(sc[0][0][i], sc[0][0][2 + i]);
        s[0][i] = from_below<8, 4>(s[0][i], sc[0][1][i]);
        s[0][i] = from_below<12, 8>(s[0][i], sc[0][1][2 + i]);
      }
    } else {
#pragma unroll
      for (int h = 0; h < kPer / 4; ++h) {
        const v4f k = *reinterpret_cast<const v4f*>(tile + l.ls + 64 * h);
        const v4f v = *reinterpret_cast<const v4f*>(tile + l.ls + 128 + 64 * h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[4 * h + i] = k[i] * scale_log2;
          vs[4 * h + i] = v[i];
#pragma unroll
          for (int r = 0; r < R; ++r)
            s[r][4 * h + i] = kPer == 4 ? from_below<8, 12>(sc[0][0][i], sc[0][1][i]) : sc[r][h][i];
        }
      }
    }
    bool odd = false;
    if (!all) {
      // what lies behind a row's last key may be anything, NaN among it
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int tok = t0 + l.tok + 16 * (i >> 2) + (i & 3);
        vs[i] = tok < L ? vs[i] : 0.f;
        odd |= !(__builtin_fabsf(vs[i]) < __builtin_inff());
#pragma unroll
        for (int r = 0; r < R; ++r) s[r][i] = tok < seen[r] ? s[r][i] * f[i] : -__builtin_inff();
        f[i] = 1.f;
      }
    }
    float sum[R];
    uint32_t pair[R][kPer / 2];
    // p = exp2(exponent(r, i)) of score i of row r
    auto probabilities = [&](auto exponent) {
      float top = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float part[kPer / 2];
#pragma unroll
        for (int i = 0; i < kPer / 2; ++i) {
          const float p0 = exp2_hw(exponent(r, 2 * i));
          const float p1 = exp2_hw(exponent(r, 2 * i + 1));
          const v2f x = {p0 * vs[2 * i], p1 * vs[2 * i + 1]};
          top = fmaxf(top, fmaxf(x[0], x[1]));
          part[i] = p0 + p1;
          pair[r][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, v2h));
        }
        sum[r] = part[0];
        if constexpr (kPer == 4) sum[r] = part[0] + part[1];
        if constexpr (kPer == 8) sum[r] = (part[0] + part[1]) + (part[2] + part[3]);
      }
      return top;
    };
    bool over = odd | (probabilities([&](int r, int i) { return __builtin_fmaf(s[r][i], f[i], -st.m[r]); }) > kTermLimit);
#pragma unroll
    for (int r = 0; r < R; ++r) over |= sum[r] > kSumLimit;
    if (__builtin_expect(__builtin_amdgcn_readfirstlane((int)(__ballot(over) != 0)) | st.far, 0)) {
      // the references move to the largest term so far
      float m[R], by[R], ref[R];
      bool rare = odd;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float em = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < kPer; ++i) em = fmaxf(em, s[r][i] * f[i] + __log2f(fmaxf(vs[i], kTinyScale)));
        m[r] = ref[r] = fmaxf(st.m[r], row_max<16 / PK>(em) - kLift);
        by[r] = exp2_hw(st.m[r] - m[r]);
        rare |= __builtin_fabsf(m[r]) >= kFar && m[r] != kUnset;
      }
      if (__builtin_expect(__builtin_amdgcn_readfirstlane((int)(__ballot(rare) != 0)) | st.far, 0))
        rare_references(s, f, vs, lifts, m, by, ref, st);
      __builtin_amdgcn_sched_barrier(0);   // (mixed with what follows, the products take more registers)
#pragma unroll
      for (int r = 0; r < R; ++r) move(r, m[r], by[r], st);
      __builtin_amdgcn_sched_barrier(0);
      (void)probabilities([&](int r, int i) { return __builtin_fmaf(s[r][i], f[i], -ref[r]); });
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      st.l[r] += sum[r];
      if constexpr (PK == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) pf[r][i] = pair[r][i];
      } else if constexpr (PK == 2) {
        pf[r] = v4u{pair[r][0], pair[r][1], from_above<8>(pair[r][0]), from_above<8>(pair[r][1])};
      } else {
        pf[r] = v4u{pair[r][0], from_above<4>(pair[r][0]), from_above<8>(pair[r][0]), from_above<12>(pair[r][0])};
      }
    }
  }

  // O^T += V^T P^T: accumulator j holds channel j of each sixteenth.  From byte
  // B of the sixteenths on.
  template <int B>
  static __device__ __forceinline__ void values(const uint32_t (*w)[kW], const v4u* pf, const Exponents& e, State& st) {
    if constexpr (B < kDB / 16) {
      uint32_t x[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        x[2 * h] = token_pair<kDB / 16, 0, B>(w[h]);
        x[2 * h + 1] = token_pair<kDB / 16, 2, B>(w[h]);
      }
      if constexpr (BITS == 4) {
        v4u lo, hi;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = less((x[i] & 0x000F000Fu) | e.lo, 1032.f);
          hi[i] = less((x[i] & 0x00F000F0u) | e.hi, 72.f);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          st.o[r][2 * B] = mma_h(lo, pf[r], st.o[r][2 * B]);
          st.o[r][2 * B + 1] = mma_h(hi, pf[r], st.o[r][2 * B + 1]);
        }
      } else {
        v4u u;
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = less(x[i] ^ e.lo, 1152.f);
#pragma unroll
        for (int r = 0; r < R; ++r) st.o[r][B] = mma_h(u, pf[r], st.o[r][B]);
      }
      values<B + 1>(w, pf, e, st);
    }
  }
  static __device__ __forceinline__ Exponents exponents() {
    return {held(KC::kExp), held(BITS == 4 ? 0x64006400u : 0x64806480u), held(0x54005400u)};
  }
};

// Query row `row` of key head h of a sequence whose first token is row0, as a
// row of [T][Hq].
__device__ __forceinline__ int64_t out_row(const AttnArgs& a, int row0, int h, uint32_t row) {
  const uint32_t i = row / (uint32_t)a.sh.G;
  return ((int64_t)row0 + i) * (a.sh.Hkv * a.sh.G) + h * a.sh.G + (row - i * a.sh.G);
}

__device__ __forceinline__ AttnSeq get_seq(const AttnArgs& a, int b) {
  if (a.q_starts) return attn_seq(a.sh, a.q_starts[b], a.q_starts[b + 1], a.kv_lens[b]);
  return attn_seq(a.sh, b * a.sh.max_q, (b + 1) * a.sh.max_q, a.kv_lens[b]);
}

// The sequence that holds a workgroup's first unit, its own first unit, the
// units of all sequences and the workgroup's share of them, found by the
// workgroup: each thread counts those of some neighbouring sequences, and a
// scan says where they begin.  b, base and sq are set if the workgroup has
// units.  red: a word per wave, then kAttnFound.
struct AttnFind {
  uint32_t total, share, base;
  int b;
  AttnSeq sq;
};
constexpr int kAttnFound = 5;
__device__ __forceinline__ AttnFind find_units(const AttnArgs& a, uint32_t workgroup, uint32_t* red) {
  constexpr int kThreads = 64 * kAttnWaves;
  const int tid = threadIdx.x, per = (a.sh.B + kThreads - 1) / kThreads, b0 = tid * per;
  AttnSeq sq = {0, 0, 0};
  uint32_t sum = 0;
  for (int b = b0; b < b0 + per && b < a.sh.B; ++b) {
    sq = get_seq(a, b);
    sum = attn_add(sum, attn_units(a.sh, sq));
  }
  uint32_t in = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(in, d, 64);
    if ((tid & 63) >= d) in = attn_add(in, o);
  }
  if ((tid & 63) == 63) red[tid >> 6] = in;
  __syncthreads();
  AttnFind f = {};
#pragma unroll
  for (int w = 0; w < kAttnWaves; ++w) {
    if (w < (tid >> 6)) in = attn_add(in, red[w]);
    f.total = attn_add(f.total, red[w]);
  }
  if (f.total > kAttnMostUnits) f.total = 0;   // contradictory starts: nothing is computed
  f.share = attn_share(f.total, a.workgroups);
  const uint32_t want = workgroup * f.share;
  if (want >= f.total) return f;
  uint32_t* const found = red + kAttnWaves;
  if (in - sum <= want && want < in) {   // one thread
    uint32_t base = in - sum;
    int b = b0;
    if (per > 1)
      for (uint32_t u; sq = get_seq(a, b), want >= base + (u = attn_units(a.sh, sq)); ++b) base += u;
    found[0] = base;
    found[1] = (uint32_t)b;
    found[2] = (uint32_t)sq.row0;
    found[3] = (uint32_t)sq.n;
    found[4] = (uint32_t)sq.L;
  }
  __syncthreads();
  f.base = __builtin_amdgcn_readfirstlane(found[0]);
  f.b = __builtin_amdgcn_readfirstlane((int)found[1]);
  f.sq.row0 = __builtin_amdgcn_readfirstlane((int)found[2]);
  f.sq.n = __builtin_amdgcn_readfirstlane((int)found[3]);
  f.sq.L = __builtin_amdgcn_readfirstlane((int)found[4]);
  return f;
}

template <bool FP16>
__device__ __forceinline__ uint32_t to16(float a, float b) {
  const v2f x = {a, b};
  if constexpr (FP16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, v2h));
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, v2b));
}

// Channels of accumulators j, j + 1 of a row: two neighbours in each of four
// sixteenths.
template <bool FP16, int D>
__device__ __forceinline__ void store_pair(const AttnArgs& a, int64_t row, int g, int j, const v4f& x, const v4f& y) {
  uint16_t* out = static_cast<uint16_t*>(a.out) + row * D;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint32_t*>(out + (4 * g + i) * (D / 16) + j) = to16<FP16>(x[i], y[i]);
}

// Places of a piece in the workspace: accumulator n of lane l of piece x, and
// a row's reference and sum.
template <int N, int ROWS>
__device__ __forceinline__ v4f* piece_o(const AttnArgs& a, uint32_t x, int n, int lane) {
  return reinterpret_cast<v4f*>(a.part) + ((int64_t)x * N + n) * 64 + lane;
}
// A segment that a workgroup begins and others go on with, for the kernel that
// joins the pieces: a record per workgroup, followers 0 where there is none.
struct AttnSplit {
  uint32_t followers, row_0, rows;
  int row0, h;
};
template <int ROWS>
__device__ __forceinline__ v2f* piece_ml(const AttnArgs& a, uint32_t x, int row) {
  return reinterpret_cast<v2f*>(a.part_ml) + (int64_t)x * ROWS + row;
}

// WHOLE: a workgroup to a segment, blockIdx.x counting sequence, row tile of
// max_q tokens, key head; otherwise the workgroup's share of all segments.
template <bool FP16, int D, int BITS, int ROWS, bool WHOLE>
__global__ __launch_bounds__((64 * Attn<FP16, D, BITS, ROWS, WHOLE>::kWaves), WHOLE ? 1 : 2) void k_attn(AttnArgs a) {
  using A = Attn<FP16, D, BITS, ROWS, WHOLE>;
  constexpr int kWaves = A::kWaves;
  constexpr int R = A::R;
  __shared__ __align__(16) uint8_t ring[A::kLdsBytes];
  float* const lds = reinterpret_cast<float*>(ring);
  __shared__ __align__(16) uint8_t query[A::kQueryLds ? A::kQueryBytes : 16];
  __shared__ float ldm[kWaves][A::kRows], ldl[kWaves][A::kRows], lifts[kWaves][A::kRows];
  __shared__ uint32_t red[kAttnWaves + kAttnFound];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, col = lane & 15;
  const int own = ROWS < 16 ? col & (ROWS - 1) : col;   // the row whose reference and sum the lane holds
  const int page = a.sh.page;
  const Exponents e = A::exponents();
  const typename A::Lane ln = A::lane_of(a, lane);
  const uint8_t* const mine = ring + wave * A::kRingBytes;
  const uint32_t mine_at = lds_addr(mine);

  uint32_t u = 0, hi = 1, base = 0, share = 0;
  int b, h_whole = 0, rt_whole = 0;
  AttnSeq sq;
  if constexpr (WHOLE) {
    const uint32_t nrt = (uint32_t)(((int64_t)a.sh.max_q * a.sh.G + ROWS - 1) / ROWS), at = blockIdx.x / (uint32_t)a.sh.Hkv;
    h_whole = (int)(blockIdx.x - at * a.sh.Hkv);
    b = (int)(at / nrt);
    rt_whole = (int)(at - b * nrt);
    sq = get_seq(a, b);
    if ((int64_t)rt_whole * ROWS >= (int64_t)sq.n * a.sh.G) return;
  } else {
    const AttnFind f = find_units(a, blockIdx.x, red);
    share = f.share;
    u = blockIdx.x * share;
    hi = u + share < f.total ? u + share : f.total;
    b = f.b;
    base = f.base;
    sq = f.sq;
  }
  AttnSplit split = {};

  while (u < hi) {
    AttnSeg sg;
    if constexpr (WHOLE) {
      sg.tiles = sg.last = attn_tiles(a.sh, sq, (uint32_t)rt_whole);
      sg.first = 0;
      sg.h = h_whole;
      sg.row_0 = (uint32_t)rt_whole * ROWS;
      sg.rows = (uint32_t)sq.n * (uint32_t)a.sh.G;
      u = hi;
    } else {
      const AttnHead hd = attn_head(a.sh, sq);
      const uint32_t units = (uint32_t)a.sh.Hkv * hd.units;
      if (u >= base + units) {
        base += units;
        sq = get_seq(a, ++b);
        continue;
      }
      sg = attn_segment(a.sh, sq, hd, u - base, hi - base);
      u += sg.units;
      if (sg.first == sg.last) continue;
    }
    const uint32_t tiles = sg.tiles, first = sg.first, last = sg.last, row_0 = sg.row_0, rows = sg.rows;
    const int h = sg.h;
    // the tokens that the first row sees, and all others then; tiles that see nothing are not computed
    const int seen_least = attn_seen(a.sh, sq, (int)(row_0 / (uint32_t)a.sh.G));
    const uint32_t row_last = row_0 + A::kRows < rows ? row_0 + A::kRows - 1 : rows - 1;
    const bool nothing = attn_seen(a.sh, sq, (int)(row_last / (uint32_t)a.sh.G)) == 0;
    const uint32_t count = nothing ? 0 : last - first;
    const uint32_t per = (count + kWaves - 1) / kWaves;
    const uint32_t t0 = first + wave * per, end = first + count, t1 = t0 + per < end ? t0 + per : end;

    // The wave's tiles one behind the other, in half tiles of 16 tokens (which
    // lie in one page).  The pages are in a register, 64 at a time, so that a page
    // id costs a lane read (and a wait for all loads before it) in place of a load
    // between the tiles.  Behind the sequence's last page the last one is read
    // again, and nothing of it counts.
    const int32_t* table = a.table + (int64_t)b * a.sh.max_pages;
    const uint32_t page_last = ((uint32_t)sq.L - 1) / (uint32_t)page;
    uint32_t n = t0 * kAttnTile / (uint32_t)page, off = t0 * kAttnTile - n * page;
    uint32_t ids = 0, ids_from = n;
    auto fetch_ids = [&] {
      ids = ids_from + lane <= page_last ? (uint32_t)table[ids_from + lane] : 0u;
    };
    if (t0 < t1) fetch_ids();
    // this lane's rows
    v4u qf[R][A::kSteps];
    int seen[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t row = row_0 + 16 * r + own, i = row / (uint32_t)a.sh.G;
      seen[r] = row < rows ? attn_seen(a.sh, sq, (int)i) : 0;
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + ((int64_t)sq.row0 + i) * a.q_stride +
                            (int64_t)(h * a.sh.G + (int)(row - i * a.sh.G)) * D + g * (D / 4);
#pragma unroll
      for (int j = 0; j < A::kSteps; ++j) {
        qf[r][j] = v4u{0u, 0u, 0u, 0u};
        if (row < rows && col < ROWS && (A::kQueryLds || t0 < t1)) qf[r][j] = *reinterpret_cast<const v4u*>(src + 8 * j);
      }
    }
    wait_loads<0>();                  // only the tiles' loads are counted from here on
    const uint32_t head_rows = (uint32_t)a.sh.Hkv * page, head = (uint32_t)h * page;
    auto next = [&] {
      const uint32_t nc = n < page_last ? n : page_last;
      if (nc - ids_from >= 64) {
        ids_from = nc;
        fetch_ids();
      }
      uint32_t pg = (uint32_t)__builtin_amdgcn_readlane((int)ids, (int)(nc - ids_from));
      if (pg >= (uint32_t)a.pages) pg = 0;   // no page of the cache: any row, and no fault
      const int64_t at = (int64_t)((uint64_t)pg * head_rows + (head + off));
      off += 16;
      if (off == (uint32_t)page) {
        off = 0;
        ++n;
      }
      return at;
    };
    uint32_t put = 0, got = 0;        // the ring's places, in bytes
    auto load = [&] {
      const int64_t at0 = next(), at1 = next();
      A::load(a, ln, at0, at1, mine_at + put);
      put = put == A::kRingBytes - A::kTileBytes ? 0 : put + A::kTileBytes;
    };
#pragma unroll
    for (int d = 0; d < A::kDepth; ++d)
      if (t0 + d < t1) load();

    typename A::State st;
    float c0[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < A::kSteps; ++j) {
        const v4u w = qf[r][j];
        float x[8];
        unpack8<FP16>(make_uint4(w[0], w[1], w[2], w[3]), x);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += x[i];
        if constexpr (BITS == 4)       // 0 4 1 5 2 6 3 7
          qf[r][j] = v4u{__builtin_amdgcn_perm(w[2], w[0], 0x05040100u), __builtin_amdgcn_perm(w[2], w[0], 0x07060302u),
                         __builtin_amdgcn_perm(w[3], w[1], 0x05040100u), __builtin_amdgcn_perm(w[3], w[1], 0x07060302u)};
      }
      c0[r] = -A::KC::kOffset * row_sum<16>(sum);
      st.m[r] = kUnset;
      st.l[r] = 0.f;
#pragma unroll
      for (int j = 0; j < A::kJ; ++j) st.o[r][j] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    st.far = false;
    const uint8_t* const ql = query + 16 * lane;
    if constexpr (A::kQueryLds) {
      // (every wave has all of it, for c0)
#pragma unroll
      for (int i = 0; i < R * A::kSteps; ++i)
        if (i % kWaves == wave) *reinterpret_cast<v4u*>(query + 1024 * i + 16 * lane) = qf[i / A::kSteps][i % A::kSteps];
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r % kWaves == wave)
          *reinterpret_cast<v4f*>(query + 1024 * (R * A::kSteps + r) + 16 * lane) = v4f{c0[r], c0[r], c0[r], c0[r]};
      __syncthreads();
    }
    for (uint32_t t = t0; t < t1; ++t) {
      // the loads of the tiles behind this one may be outstanding
      const uint32_t behind = t1 - 1 - t;
      if (A::kDepth > 3 && behind >= 3) wait_loads<(A::kDepth > 3 ? 3 * A::kLoads : 0)>();
      else if (A::kDepth > 2 && behind >= 2) wait_loads<(A::kDepth > 2 ? 2 * A::kLoads : 0)>();
      else if (behind >= 1) wait_loads<A::kLoads>();
      else wait_loads<0>();
      const uint8_t* tile = mine + got;
      v4f s[R][2];
      v4u pf[R];
      A::scores(tile, ln, qf, ql, c0, e, s);
      A::softmax(tile, ln, s, a.scale_log2, (int)t * kAttnTile, attn_tile_full(t, seen_least), sq.L, seen,
                 lifts[wave], st, pf);
      uint32_t w[2][A::kW];
      A::values_of(tile, ln, 0, w[0]);
      A::values_of(tile, ln, 1, w[1]);
      if (t + A::kDepth < t1) {
        wait_lds_reads();
        load();
      }
      A::template values<0>(w, pf, e, st);
      got = got == A::kRingBytes - A::kTileBytes ? 0 : got + A::kTileBytes;
    }

    // fp32 holds the sums without the lifts
    if (__builtin_expect(st.far, 0)) {
#pragma unroll
      for (int r = 0; r < R; ++r) A::move(r, st.m[r], exp2_hw(-lifts[wave][16 * r + own]), st);
    }

    // the waves join: common references, then the sums through LDS
    const bool whole = WHOLE || (first == 0 && last == tiles);
    const uint32_t piece = attn_place(blockIdx.x, first == 0);
    if (first == 0 && !whole) split = {attn_followers(tiles, last, share), row_0, rows, sq.row0, h};
    float fw[R], M[R], Ls[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      st.l[r] = row_sum<16 / A::PK>(st.l[r]);
      if (g == 0 && col < ROWS) {
        ldm[wave][16 * r + col] = st.m[r];
        ldl[wave][16 * r + col] = st.l[r];
      }
    }
    __syncthreads();   // and every wave is through with its ring
#pragma unroll
    for (int r = 0; r < R; ++r) {
      M[r] = ldm[0][16 * r + own];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) M[r] = fmaxf(M[r], ldm[w][16 * r + own]);
      Ls[r] = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) Ls[r] += ldl[w][16 * r + own] * exp2_hw(ldm[w][16 * r + own] - M[r]);
      fw[r] = exp2_hw(st.m[r] - M[r]);
      if (whole) fw[r] = Ls[r] == 0.f ? 0.f : fw[r] / Ls[r];
    }
    constexpr int kAcc = R * A::kJ;
#pragma unroll
    for (int n0 = 0; n0 < kAcc; n0 += A::kRound) {
      constexpr int kN = kAcc < A::kRound ? kAcc : A::kRound;
      if (n0) __syncthreads();
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        const int r = (n0 + n) / A::kJ, j = (n0 + n) % A::kJ;
        *reinterpret_cast<v4f*>(&lds[((wave * A::kRound + n) * 64 + lane) * 4]) = st.o[r][j] * fw[r];
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < kN; n += 2 * kWaves) {
        const int nn = n + 2 * wave;
        if (kN < 2 * kWaves && nn >= kN) continue;
        v4f sum[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sum[e] = *reinterpret_cast<const v4f*>(&lds[((nn + e) * 64 + lane) * 4]);
#pragma unroll
          for (int w = 1; w < kWaves; ++w)
            sum[e] += *reinterpret_cast<const v4f*>(&lds[((w * A::kRound + nn + e) * 64 + lane) * 4]);
        }
        const int r = (n0 + nn) / A::kJ, j = (n0 + nn) % A::kJ;
        const uint32_t row = row_0 + 16 * r + col;
        if (row < rows && col < ROWS) {
          if (whole) {
            store_pair<FP16, D>(a, out_row(a, sq.row0, h, row), g, j, sum[0], sum[1]);
          } else {
            *piece_o<kAcc, A::kRows>(a, piece, n0 + nn, lane) = sum[0];
            *piece_o<kAcc, A::kRows>(a, piece, n0 + nn + 1, lane) = sum[1];
          }
        }
      }
    }
    if (wave == 0 && g == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t row = row_0 + 16 * r + col;
        if (row < rows && col < ROWS) {
          if (!whole) *piece_ml<A::kRows>(a, piece, 16 * r + col) = v2f{M[r], Ls[r]};
          else if (a.lse) a.lse[out_row(a, sq.row0, h, row)] = log_sum(M[r], Ls[r]);
        }
      }
    }
    __syncthreads();   // LDS is free for the next segment
  }
  if (!WHOLE && threadIdx.x == 0) static_cast<AttnSplit*>(a.splits)[blockIdx.x] = split;
}

// The segments that more than one workgroup holds: workgroup w joins the one
// that workgroup w began, if there is one.  SPREAD: a workgroup to an
// accumulator, whose waves take turns at the pieces and join in LDS; otherwise
// a wave to every fourth accumulator, with all pieces in order.  Bound by the
// latency of its loads: traced, 64 pieces of each of 8 segments 7.1 us spread, the
// pieces of 512 segments 5.0 us in order.
template <bool FP16, int D, int ROWS, bool SPREAD>
__global__ __launch_bounds__(SPREAD ? 512 : 256) void k_attn_join(AttnArgs a) {
  constexpr int kJ = D / 16, kAcc = (ROWS > 16 ? ROWS / 16 : 1) * kJ, kWaves = SPREAD ? 8 : 4;
  const AttnSplit sp = static_cast<const AttnSplit*>(a.splits)[blockIdx.x];
  if (sp.followers == 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, col = lane & 15;
  __shared__ v4f lo[SPREAD ? kWaves : 1][64];
  __shared__ v2f lml[SPREAD ? kWaves : 1][64];

  const int n = SPREAD ? (int)blockIdx.y : (int)blockIdx.y * kWaves + wave;
  const int r = n / kJ, j = n % kJ;
  const uint32_t row = sp.row_0 + 16 * r + col;
  const bool there = row < sp.rows && col < ROWS;
  float M = kUnset, Ls = 0.f;
  v4f o = {0.f, 0.f, 0.f, 0.f};
  if (there) {
#pragma unroll 8
    for (uint32_t w = SPREAD ? wave : 0; w <= sp.followers; w += SPREAD ? kWaves : 1) {
      const uint32_t x = attn_place(blockIdx.x + w, w == 0);
      const v2f ml = *piece_ml<ROWS>(a, x, 16 * r + col);
      const v4f po = *piece_o<kAcc, ROWS>(a, x, n, lane);
      const float m = fmaxf(M, ml[0]), f0 = exp2_hw(M - m), f1 = exp2_hw(ml[0] - m);
      o = o * f0 + po * f1;
      Ls = Ls * f0 + ml[1] * f1;
      M = m;
    }
  }
  if constexpr (SPREAD) {
    lo[wave][lane] = o;
    lml[wave][lane] = v2f{M, Ls};
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
      const v2f ml = lml[w][lane];
      const float m = fmaxf(M, ml[0]), f0 = exp2_hw(M - m), f1 = exp2_hw(ml[0] - m);
      o = o * f0 + lo[w][lane] * f1;
      Ls = Ls * f0 + ml[1] * f1;
      M = m;
    }
  }
  if (!there) return;
  const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
  const int64_t orow = out_row(a, sp.row0, sp.h, row);
  uint16_t* out = static_cast<uint16_t*>(a.out) + orow * D;
#pragma unroll
  for (int i = 0; i < 4; ++i) out[(4 * g + i) * kJ + j] = (uint16_t)to16<FP16>(o[i] * inv, 0.f);
  if (a.lse && j == 0 && g == 0) a.lse[orow] = log_sum(M, Ls);
}

template <bool FP16, int D, int BITS, int ROWS>
hipError_t attn_go(const AttnArgs& a, hipStream_t st) {
  const int64_t segments = (int64_t)a.sh.B * a.sh.Hkv * (((int64_t)a.sh.max_q * a.sh.G + ROWS - 1) / ROWS);
  if constexpr (ROWS <= 16) {
    if (attn_takes_whole(a.sh, segments, D * BITS / 8)) {
      hipLaunchKernelGGL((k_attn<FP16, D, BITS, ROWS, true>), dim3((unsigned)segments),
                         dim3(64 * attn_whole_waves(D * BITS / 8)), 0, st, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((k_attn<FP16, D, BITS, ROWS, false>), dim3((unsigned)a.workgroups), dim3(64 * kAttnWaves), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // Many pieces to a segment where there are few segments.  Measured, us of a
  // call spread and in order: 8 segments of 8192 tokens 14.9 and 15.5, of 131072
  // 38.1 and 38.9, 64 of up to 4000 16.3 and 17.0; 512 of up to 16384 101.2 and
  // 99.0, 2048 of up to 1000 50.4 and 48.6.
  constexpr int kAcc = (ROWS > 16 ? ROWS / 16 : 1) * D / 16;
  if (segments * 4 <= a.workgroups)
    hipLaunchKernelGGL((k_attn_join<FP16, D, ROWS, true>),
                       dim3((unsigned)a.workgroups - 1, kAcc), dim3(512), 0, st, a);
  else
    hipLaunchKernelGGL((k_attn_join<FP16, D, ROWS, false>), dim3((unsigned)a.workgroups - 1, kAcc / 4), dim3(256), 0, st, a);
  return hipGetLastError();
}

template <bool FP16, int D, int BITS>
hipError_t attn_rows(const AttnArgs& a, hipStream_t st) {
  switch (a.sh.rows) {
    case 4: return attn_go<FP16, D, BITS, 4>(a, st);
    case 8: return attn_go<FP16, D, BITS, 8>(a, st);
    case 16: return attn_go<FP16, D, BITS, 16>(a, st);
    default:
      if constexpr (D < 256)
        return a.sh.rows == 32 ? attn_go<FP16, D, BITS, 32>(a, st) : attn_go<FP16, D, BITS, 64>(a, st);
      return hipErrorInvalidValue;
  }
}

template <bool FP16, int D>
hipError_t attn_pick(const AttnArgs& a, int bits, hipStream_t st) {
  return bits == 4 ? attn_rows<FP16, D, 4>(a, st) : attn_rows<FP16, D, 8>(a, st);
}

}  // namespace

// Rows to a row tile, workgroups and workspace of a call.  A larger tile takes
// the codes apart for more rows at once, smaller ones are more and shorter
// segments.  Measured, us with 16, 32 and 64 rows (query rows of the call in
// brackets): 4 tokens of 8 requests (768) 21, 25, -; 64 tokens on 4000 (2048)
// 28, 30, 40; 16 tokens of 8 requests (4096) 39, 38, 46; 256 tokens on 4000
// (8192) 55, 52, 61; 16 tokens of 64 requests (32768) 105, 74, 75; prompts'
// pieces and single tokens (53000) 224, 167, 164; 2048 tokens on 8192 (65536)
// 592, 387, 315.  256 channels leave registers for 16 rows only: 4 tokens of
// 64 requests (2560) 63, 92, -.
// 512 workgroups: two to a CU stream as fast as four (64 sequences of 8192:
// 107 us with 512, 112 with 1024), and leave half the pieces.  Two do not fit with
// 8 bits and 256 channels (133 KB of LDS) or 128 channels in 64 rows (91 KB):
// these run in two rounds (2048 tokens on 8192 in 8 bits 551 to 557 us; one round of 256 was
// not measured).
int64_t attn_workspace(AttnArgs* a, int64_t D, void* ws) {
  const int64_t rows = (int64_t)a->sh.max_q * a->sh.G, all = (int64_t)a->sh.T * a->sh.Hkv * a->sh.G;
  a->sh.rows = rows <= 4 ? 4 : rows <= 8 ? 8 : rows <= 16 || D == 256 || all < 4096 ? 16 : rows <= 32 || all < 40000 ? 32 : 64;
  a->workgroups = 512;
  // (room for the largest tile of these heads: the size goes by them alone)
  const int64_t pieces = 2 * (int64_t)a->workgroups, kept = rows <= 16 || D == 256 ? 16 : rows <= 32 ? 32 : 64;
  const int64_t o = pieces * kept * D * 4, ml = o + pieces * kept * 8;
  a->part = static_cast<float*>(ws);
  a->part_ml = ws ? reinterpret_cast<float*>(static_cast<char*>(ws) + o) : nullptr;
  a->splits = ws ? static_cast<char*>(ws) + ml : nullptr;
  return ml + (int64_t)a->workgroups * sizeof(AttnSplit);
}

hipError_t launch_attn(const AttnArgs& a, bool fp16, int bits, int D, hipStream_t st) {
  if (fp16) {
    if (D == 64) return attn_pick<true, 64>(a, bits, st);
    if (D == 128) return attn_pick<true, 128>(a, bits, st);
    return attn_pick<true, 256>(a, bits, st);
  }
  if (D == 64) return attn_pick<false, 64>(a, bits, st);
  if (D == 128) return attn_pick<false, 128>(a, bits, st);
  return attn_pick<false, 256>(a, bits, st);
}

}  // namespace w8
