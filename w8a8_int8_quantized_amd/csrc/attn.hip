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
// No operand passes through LDS.
//
// Codes to 16-bit floats: OR an exponent on top of the code bits in place,
// which gives 2^k + code + offset exactly.  For the keys the constant is not
// subtracted from each but once from the sum: the accumulators start at
// -(2^k + offset) * sum_d q[d].  For the values it is subtracted (exact in
// fp16): a running sum over a long cache must not carry an offset that is
// larger than its result.
//
// Softmax: m is a reference that a row's scores may pass by a factor of 32
// before it moves (the largest p vs / vref is looked at, one compare a tile),
// so the accumulators are seldom rescaled.  p vs goes into the second product
// as fp16, scaled by 1024 / vref (vref: the largest vs so far): half a step is
// 2^-11 of the probability, and what lies 2^-24 below the largest term is
// rounded to that.  m, l and all sums are fp32.
//
// Work is shared out in equal runs of 32-token tiles over all sequences and
// heads (attn_plan.h); the waves of a workgroup take parts of a segment's run
// and join in LDS; a segment that more than one workgroup holds is joined by
// a second kernel, in order, so results do not depend on timing.
#include "attn_plan.h"
#include "common.h"
#include "launch.h"

namespace w8 {
namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

constexpr float kUnset = -1e30f;     // a reference before the first score
constexpr float kLift = 1024.f;      // what the largest p vs / vref is scaled to
constexpr float kLimit = 32768.f;    // and what it may grow to: fp16 ends at 65504
constexpr float kLn2 = 0.693147180559945309f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Across the four lanes of a row (lane ^ 16, lane ^ 32).
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// N dwords of a lane from a 4 N-byte aligned address.
template <int N>
__device__ __forceinline__ void load_words(uint32_t* w, const uint8_t* p) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const v4u v = *reinterpret_cast<const v4u*>(p + 16 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
    }
  } else {
    const v2u v = *reinterpret_cast<const v2u*>(p);
    w[0] = v[0];
    w[1] = v[1];
  }
}

// ------------------------------------------------------------ codes to floats
// The key operand of one matrix instruction, 8 channels of a lane's quarter.
// 4 bits: channels in the order 0 4 1 5 2 6 3 7 (the query's operand has the
// same), value 128 + n (bf16) or 64 + n (fp16), n = code + 8.  8 bits: in
// order, value code + 128 (bf16) or 1024 + code + 128 (fp16).
template <bool FP16, int BITS>
struct KeyCodes {
  static constexpr float kOffset = BITS == 4 ? (FP16 ? 72.f : 136.f) : (FP16 ? 1152.f : 128.f);
  static __device__ __forceinline__ v4u operand(const uint32_t* w) {
    v4u r;
    if constexpr (BITS == 4 && FP16) {
      r[0] = ((w[0] << 4) & 0x00F000F0u) | 0x54005400u;
      r[1] = (w[0] & 0x00F000F0u) | 0x54005400u;
      r[2] = ((w[0] >> 4) & 0x00F000F0u) | 0x54005400u;
      r[3] = ((w[0] >> 8) & 0x00F000F0u) | 0x54005400u;
    } else if constexpr (BITS == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = ((w[0] >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t u = w[i] ^ 0x80808080u;
        if constexpr (FP16) {
          r[2 * i] = __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u);
          r[2 * i + 1] = __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u);
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
template <bool FP16, int D, int BITS, int R>
struct Attn {
  static constexpr int kDB = D * BITS / 8;          // bytes of a token's codes
  static constexpr int kW = kDB / 16;               // dwords of a lane per half tile, keys or values
  static constexpr int kSteps = D / 32;             // matrix instructions per half tile of S^T
  static constexpr int kJ = D / 16;                 // channels of a sixteenth: accumulators of O^T
  static constexpr int kRows = 16 * R;
  static constexpr int kRegs = R * kJ * 4;          // accumulator registers of a lane
  static constexpr int kRound = 8;                  // accumulators (of 4) per round through LDS
  static constexpr int kLdsFloats = kAttnWaves * kRound * 4 * 64;
  using KC = KeyCodes<FP16, BITS>;

  struct Tile {
    uint32_t k[2][kW], v[2][kW];
    v4f ks[2], vs[2];
  };
  struct State {
    v4f o[R][kJ];
    float m[R], l[R], vref;
  };

  static __device__ __forceinline__ v4f mma(const v4u& a, const v4u& b, const v4f& c) {
    if constexpr (FP16)
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0,
                                                     0);
  }

  // base: the half tiles' first token as a row of [pages][Hkv][page].
  static __device__ __forceinline__ void load(const AttnArgs& a, const int64_t* base, int lane, Tile& t) {
    const uint32_t m = lane & 15, g = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      load_words<kW>(t.k[h], a.k + base[h] * kDB + (m * kDB + g * (kDB / 4)));
      t.ks[h] = *reinterpret_cast<const v4f*>(a.ks + base[h] + 4 * g);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      load_words<kW>(t.v[h], a.v + base[h] * kDB + (g * 4 * kDB + m * (kDB / 4)));
      t.vs[h] = *reinterpret_cast<const v4f*>(a.vs + base[h] + 4 * g);
    }
  }

  // Token t0 .. t0 + 31 of the sequence.  seen: the keys that the lane's rows
  // see; all: whether every row sees the whole tile.
  static __device__ __forceinline__ void compute(const Tile& t, const v4u (*qf)[kSteps], const float* c0,
                                                 float scale_log2, int t0, bool all, int L, const int* seen, int lane,
                                                 State& st) {
    const int g = lane >> 4;
    v4f s[R][2], vs[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int r = 0; r < R; ++r) s[r][h] = v4f{c0[r], c0[r], c0[r], c0[r]};
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const v4u ko = KC::operand(t.k[h] + j * (BITS / 4));
#pragma unroll
        for (int r = 0; r < R; ++r) s[r][h] = mma(ko, qf[r][j], s[r][h]);
      }
      const v4f f = t.ks[h] * scale_log2;
#pragma unroll
      for (int r = 0; r < R; ++r) s[r][h] *= f;
      vs[h] = t.vs[h];
    }
    if (!all) {
      // what lies behind a row's last key may be anything, NaN among it
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = t0 + 16 * h + 4 * g + i;
          vs[h][i] = tok < L ? vs[h][i] : 0.f;
#pragma unroll
          for (int r = 0; r < R; ++r) s[r][h][i] = tok < seen[r] ? s[r][h][i] : -__builtin_inff();
        }
    }
    float c = kLift / st.vref;
    float p[R][8], pv[R][8], top = 0.f;
    auto probabilities = [&] {
      top = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          p[r][i] = exp2_hw(s[r][i >> 2][i & 3] - st.m[r]);
          pv[r][i] = p[r][i] * (vs[i >> 2][i & 3] * c);
          top = fmaxf(top, pv[r][i]);
        }
    };
    probabilities();
    if (__ballot(top > kLimit || st.m[0] == kUnset) != 0) {
      // the references move to the largest so far
      float vm = st.vref;
#pragma unroll
      for (int i = 0; i < 8; ++i) vm = fmaxf(vm, vs[i >> 2][i & 3]);
      vm = row_max(vm);
      const float fv = st.vref / vm;
      st.vref = vm;
      c = kLift / vm;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float sm = st.m[r];
#pragma unroll
        for (int i = 0; i < 8; ++i) sm = fmaxf(sm, s[r][i >> 2][i & 3]);
        sm = row_max(sm);
        const float f = exp2_hw(st.m[r] - sm);
        st.m[r] = sm;
        st.l[r] *= f;
#pragma unroll
        for (int j = 0; j < kJ; ++j) st.o[r][j] *= f * fv;
      }
      probabilities();
    }
    v4u pf[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const v2f x = {pv[r][2 * i], pv[r][2 * i + 1]};
        pf[r][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, v2h));
      }
      st.l[r] += ((p[r][0] + p[r][1]) + (p[r][2] + p[r][3])) + ((p[r][4] + p[r][5]) + (p[r][6] + p[r][7]));
    }
    values(t, pf, st);
  }

  // O^T += V^T P^T: accumulator j holds channel j of each sixteenth.
  static __device__ __forceinline__ void values(const Tile& t, const v4u* pf, State& st) {
    value_bytes<0>(t, pf, st);
  }

  template <int B>
  static __device__ __forceinline__ void value_bytes(const Tile& t, const v4u* pf, State& st) {
    if constexpr (B < kDB / 16) {
      uint32_t x[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        x[2 * h] = token_pair<kDB / 16, 0, B>(t.v[h]);
        x[2 * h + 1] = token_pair<kDB / 16, 2, B>(t.v[h]);
      }
      if constexpr (BITS == 4) {
        v4u lo, hi;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = less((x[i] & 0x000F000Fu) | 0x64006400u, 1032.f);
          hi[i] = less((x[i] & 0x00F000F0u) | 0x54005400u, 72.f);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          st.o[r][2 * B] = mma_h(lo, pf[r], st.o[r][2 * B]);
          st.o[r][2 * B + 1] = mma_h(hi, pf[r], st.o[r][2 * B + 1]);
        }
      } else {
        v4u u;
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = less((x[i] ^ 0x00800080u) | 0x64006400u, 1152.f);
#pragma unroll
        for (int r = 0; r < R; ++r) st.o[r][B] = mma_h(u, pf[r], st.o[r][B]);
      }
      value_bytes<B + 1>(t, pf, st);
    }
  }
  static __device__ __forceinline__ v4f mma_h(const v4u& a, const v4u& b, const v4f& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  }
};

// Query row `row` of a sequence and key head h, as a row of [T][Hq].
__device__ __forceinline__ int64_t out_row(const AttnArgs& a, const AttnSeq& s, int h, uint32_t row) {
  const uint32_t i = row / (uint32_t)a.sh.G;
  return ((int64_t)s.row0 + i) * (a.sh.Hkv * a.sh.G) + h * a.sh.G + (row - i * a.sh.G);
}

__device__ __forceinline__ AttnSeq get_seq(const AttnArgs& a, int b) {
  if (a.q_starts) return attn_seq(a.sh, a.q_starts[b], a.q_starts[b + 1], a.kv_lens[b]);
  return attn_seq(a.sh, b * a.sh.max_q, (b + 1) * a.sh.max_q, a.kv_lens[b]);
}

// The sequence that holds a workgroup's first unit (workgroup x of
// a.workgroups, with shares as attn_share gives them), its own first unit, and
// the units of all sequences, found by a workgroup of NT threads: each counts
// those of some neighbouring sequences, and a scan says where they begin.  b
// and base are set if the workgroup has units.
struct AttnFind {
  uint32_t total, share, base;
  int b;
};
template <int NT>
__device__ __forceinline__ AttnFind find_units(const AttnArgs& a, uint32_t x, uint32_t* red) {
  const int tid = threadIdx.x, per = (a.sh.B + NT - 1) / NT, b0 = tid * per;
  uint32_t sum = 0;
  for (int b = b0; b < b0 + per && b < a.sh.B; ++b) sum += attn_units(a.sh, get_seq(a, b));
  uint32_t in = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(in, d, 64);
    if ((tid & 63) >= d) in += o;
  }
  if ((tid & 63) == 63) red[tid >> 6] = in;
  __syncthreads();
  AttnFind f = {0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) {
    if (w < (tid >> 6)) in += red[w];
    f.total += red[w];
  }
  f.share = attn_share(f.total, a.workgroups);
  const uint32_t want = x * f.share;
  if (want >= f.total) return f;
  if (in - sum <= want && want < in) {   // one thread
    uint32_t base = in - sum;
    int b = b0;
    for (uint32_t u; want >= base + (u = attn_units(a.sh, get_seq(a, b))); ++b) base += u;
    red[NT / 64] = base;
    red[NT / 64 + 1] = (uint32_t)b;
  }
  __syncthreads();
  f.base = __builtin_amdgcn_readfirstlane(red[NT / 64]);
  f.b = __builtin_amdgcn_readfirstlane((int)red[NT / 64 + 1]);
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
template <int ROWS>
__device__ __forceinline__ v2f* piece_ml(const AttnArgs& a, uint32_t x, int row) {
  return reinterpret_cast<v2f*>(a.part_ml) + (int64_t)x * ROWS + row;
}

template <bool FP16, int D, int BITS, int R>
__global__ __launch_bounds__(64 * kAttnWaves, D == 256 || (D == 128 && R == 2) ? 1 : 2) void k_attn(AttnArgs a) {
  using A = Attn<FP16, D, BITS, R>;
  __shared__ __align__(16) float lds[A::kLdsFloats];
  __shared__ float ldm[kAttnWaves][A::kRows], ldl[kAttnWaves][A::kRows];
  __shared__ uint32_t red[kAttnWaves + 2];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, col = lane & 15;
  const int page = a.sh.page;

  const AttnFind f = find_units<64 * kAttnWaves>(a, blockIdx.x, red);
  const uint32_t share = f.share;
  const uint32_t lo = blockIdx.x * share, hi = lo + share < f.total ? lo + share : f.total;
  if (lo >= f.total) return;

  int b = f.b;
  uint32_t base = f.base;
  for (uint32_t u = lo; u < hi;) {
    const AttnSeq sq = get_seq(a, b);
    const uint32_t units = attn_units(a.sh, sq);
    if (u >= base + units) {
      base += units;
      ++b;
      continue;
    }
    const AttnSeg sg = attn_segment(a.sh, sq, u - base, hi - base);
    const uint32_t tiles = sg.tiles, first = sg.first, last = sg.last, row_0 = sg.row_0, rows = sg.rows;
    const int h = sg.h;
    const uint32_t row_last = row_0 + A::kRows < rows ? row_0 + A::kRows - 1 : rows - 1;
    // tiles that the last row sees, and tokens that the first does
    const int seen_most = attn_seen(a.sh, sq, (int)(row_last / (uint32_t)a.sh.G));
    const int seen_least = attn_seen(a.sh, sq, (int)(row_0 / (uint32_t)a.sh.G));
    const uint32_t end_seen = (uint32_t)(seen_most + kAttnTile - 1) / kAttnTile;
    const uint32_t end = last < end_seen ? last : end_seen;
    const uint32_t count = end > first ? end - first : 0;
    const uint32_t per = (count + kAttnWaves - 1) / kAttnWaves;
    const uint32_t t0 = first + wave * per, t1 = t0 + per < end ? t0 + per : end;

    // this lane's rows
    v4u qf[R][A::kSteps];
    float c0[R];
    int seen[R];
    typename A::State st;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t row = row_0 + 16 * r + col;
      const bool there = row < rows;
      const uint32_t i = row / (uint32_t)a.sh.G;
      seen[r] = there ? attn_seen(a.sh, sq, (int)i) : 0;
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + ((int64_t)sq.row0 + i) * a.q_stride +
                            (int64_t)(h * a.sh.G + (int)(row - i * a.sh.G)) * D + g * (D / 4);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < A::kSteps; ++j) {
        v4u w = {0u, 0u, 0u, 0u};
        if (there) w = *reinterpret_cast<const v4u*>(src + 8 * j);
        float x[8];
        unpack8<FP16>(make_uint4(w[0], w[1], w[2], w[3]), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += x[e];
        if constexpr (BITS == 4) {   // 0 4 1 5 2 6 3 7
          qf[r][j][0] = __builtin_amdgcn_perm(w[2], w[0], 0x05040100u);
          qf[r][j][1] = __builtin_amdgcn_perm(w[2], w[0], 0x07060302u);
          qf[r][j][2] = __builtin_amdgcn_perm(w[3], w[1], 0x05040100u);
          qf[r][j][3] = __builtin_amdgcn_perm(w[3], w[1], 0x07060302u);
        } else {
          qf[r][j] = w;
        }
      }
      c0[r] = -A::KC::kOffset * row_sum(sum);
      st.m[r] = kUnset;
      st.l[r] = 0.f;
#pragma unroll
      for (int j = 0; j < A::kJ; ++j) st.o[r][j] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    st.vref = 1e-30f;

    const int32_t* table = a.table + (int64_t)b * a.sh.max_pages;
    auto where = [&](uint32_t t, int64_t* at) {
      const uint32_t tok = t * kAttnTile;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        // a half without tokens takes the first half's page: nothing of it counts
        const uint32_t tk = tok + 16 * x < (uint32_t)sq.L ? tok + 16 * x : tok;
        const uint32_t n = tk / (uint32_t)page;
        uint32_t pg = (uint32_t)table[n];
        if (pg >= (uint32_t)a.pages) pg = 0;   // no page of the cache: any row, and no fault
        at[x] = ((int64_t)pg * a.sh.Hkv + h) * page + (tk - n * page);
      }
    };
    if (t0 < t1) {
      typename A::Tile x, y;
      int64_t at[2];
      where(t0, at);
      A::load(a, at, lane, x);
      for (uint32_t t = t0; t < t1; t += 2) {
        if (t + 1 < t1) {
          where(t + 1, at);
          A::load(a, at, lane, y);
        }
        A::compute(x, qf, c0, a.scale_log2, (int)t * kAttnTile, (int)(t + 1) * kAttnTile <= seen_least, sq.L, seen,
                   lane, st);
        if (t + 1 < t1) {
          if (t + 2 < t1) {
            where(t + 2, at);
            A::load(a, at, lane, x);
          }
          A::compute(y, qf, c0, a.scale_log2, (int)(t + 1) * kAttnTile, (int)(t + 2) * kAttnTile <= seen_least, sq.L,
                     seen, lane, st);
        }
      }
    }

    // the waves join: common references, then the sums through LDS
    const bool whole = first == 0 && last == tiles;
    const uint32_t piece = attn_place(blockIdx.x, u - first, share);
    float fw[R], M[R], Ls[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      st.l[r] = row_sum(st.l[r]);
      if (g == 0) {
        ldm[wave][16 * r + col] = st.m[r];
        ldl[wave][16 * r + col] = st.l[r];
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      M[r] = ldm[0][16 * r + col];
#pragma unroll
      for (int w = 1; w < kAttnWaves; ++w) M[r] = fmaxf(M[r], ldm[w][16 * r + col]);
      Ls[r] = 0.f;
#pragma unroll
      for (int w = 0; w < kAttnWaves; ++w) Ls[r] += ldl[w][16 * r + col] * exp2_hw(ldm[w][16 * r + col] - M[r]);
      fw[r] = exp2_hw(st.m[r] - M[r]) * (st.vref * (1.f / kLift));
      if (whole) fw[r] = Ls[r] > 0.f ? fw[r] / Ls[r] : 0.f;
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
      for (int n = 0; n < kN; n += 2 * kAttnWaves) {
        const int nn = n + 2 * wave;
        if (kN < 2 * kAttnWaves && nn >= kN) continue;
        v4f sum[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sum[e] = *reinterpret_cast<const v4f*>(&lds[((nn + e) * 64 + lane) * 4]);
#pragma unroll
          for (int w = 1; w < kAttnWaves; ++w)
            sum[e] += *reinterpret_cast<const v4f*>(&lds[((w * A::kRound + nn + e) * 64 + lane) * 4]);
        }
        const int r = (n0 + nn) / A::kJ, j = (n0 + nn) % A::kJ;
        const uint32_t row = row_0 + 16 * r + col;
        if (row < rows) {
          if (whole) {
            store_pair<FP16, D>(a, out_row(a, sq, h, row), g, j, sum[0], sum[1]);
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
        if (row < rows) {
          if (!whole) *piece_ml<A::kRows>(a, piece, 16 * r + col) = v2f{M[r], Ls[r]};
          else if (a.lse) a.lse[out_row(a, sq, h, row)] = Ls[r] > 0.f ? M[r] * kLn2 + __logf(Ls[r]) : -__builtin_inff();
        }
      }
    }
    __syncthreads();   // LDS is free for the next segment
    u += last - first;
  }
}

// Segments that more than one workgroup holds: workgroup w joins the one that
// w is the first to hold and w + 1 goes on with, if there is one.  Each wave
// takes accumulators of its own and all pieces in order.
template <bool FP16, int D, int R>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  constexpr int kJ = D / 16, kAcc = R * kJ, kRows = 16 * R;
  __shared__ uint32_t red[6];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, col = lane & 15;
  const AttnFind f = find_units<256>(a, blockIdx.x + 1, red);
  const uint32_t share = f.share;
  const uint32_t border = (blockIdx.x + 1) * share;     // the first unit of the next workgroup
  if (border >= f.total) return;
  const uint32_t base = f.base;
  const AttnSeq sq = get_seq(a, f.b);
  const AttnSeg sg = attn_segment(a.sh, sq, border - base, border - base + 1);
  const uint32_t s0 = border - sg.first;               // the segment's first unit
  if (s0 == border || s0 < blockIdx.x * share) return;  // begins there, or with an earlier workgroup
  const uint32_t wl = (s0 + sg.tiles - 1) / share;      // the last workgroup that holds some of it
  const uint32_t row_0 = sg.row_0, rows = sg.rows;

  for (int n = wave; n < kAcc; n += 4) {
    const int r = n / kJ, j = n % kJ;
    const uint32_t row = row_0 + 16 * r + col;
    if (row >= rows) continue;
    float M = kUnset, Ls = 0.f;
    v4f o = {0.f, 0.f, 0.f, 0.f};
    for (uint32_t w = blockIdx.x; w <= wl; ++w) {
      const uint32_t x = attn_place(w, s0, share);
      const v2f ml = *piece_ml<kRows>(a, x, 16 * r + col);
      const v4f po = *piece_o<kAcc, kRows>(a, x, n, lane);
      const float m = fmaxf(M, ml[0]), f0 = exp2_hw(M - m), f1 = exp2_hw(ml[0] - m);
      o = o * f0 + po * f1;
      Ls = Ls * f0 + ml[1] * f1;
      M = m;
    }
    const float inv = Ls > 0.f ? 1.f / Ls : 0.f;
    const int64_t orow = out_row(a, sq, sg.h, row);
    uint16_t* out = static_cast<uint16_t*>(a.out) + orow * D;
#pragma unroll
    for (int i = 0; i < 4; ++i) out[(4 * g + i) * kJ + j] = (uint16_t)to16<FP16>(o[i] * inv, 0.f);
    if (a.lse && j == 0 && g == 0) a.lse[orow] = Ls > 0.f ? M * kLn2 + __logf(Ls) : -__builtin_inff();
  }
}

template <bool FP16, int D, int BITS, int R>
hipError_t attn_go(const AttnArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((k_attn<FP16, D, BITS, R>), dim3((unsigned)a.workgroups), dim3(64 * kAttnWaves), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.workgroups == 1) return e;
  hipLaunchKernelGGL((k_attn_join<FP16, D, R>), dim3((unsigned)a.workgroups - 1), dim3(256), 0, st, a);
  return hipGetLastError();
}

template <bool FP16, int D>
hipError_t attn_pick(const AttnArgs& a, int bits, hipStream_t st) {
  if constexpr (D < 256) {
    if (a.sh.rows == 32) return bits == 4 ? attn_go<FP16, D, 4, 2>(a, st) : attn_go<FP16, D, 8, 2>(a, st);
  }
  return bits == 4 ? attn_go<FP16, D, 4, 1>(a, st) : attn_go<FP16, D, 8, 1>(a, st);
}

}  // namespace

// Rows to a row tile, workgroups and workspace of a call.
int64_t attn_workspace(AttnArgs* a, int64_t D, void* ws) {
  a->sh.rows = (int64_t)a->sh.max_q * a->sh.G <= 16 || D == 256 ? 16 : 32;
  a->workgroups = 1024;
  const int64_t pieces = 2 * (int64_t)a->workgroups;
  const int64_t o = pieces * a->sh.rows * D * 4;
  a->part = static_cast<float*>(ws);
  a->part_ml = ws ? reinterpret_cast<float*>(static_cast<char*>(ws) + o) : nullptr;
  return o + pieces * a->sh.rows * 8;
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
