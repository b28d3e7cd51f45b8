// The router of a mixture-of-experts layer (gfx950): scores, the choice of
// each token's experts, and their weights.
//
//   s = softmax(l) or 1 / (1 + exp(-l));   c = s + bias
//   the topk largest c of the experts whose group stays; w = s, renormalised
//
// That DeepSeek's feed-forward layers are mixtures of experts is stated on
// "FP8 vs INT8 quantisation for DeepSeek", section 1.2.
//
// Scores and choice are computed in 64 bits: the choice is a comparison of
// numbers that may lie anywhere near each other, and in 32 bits the rounding
// of exp and of the sum would decide between experts whose logits differ.  In
// 64 bits it does so only where scores saturate (sigmoid of logits from about
// 37 up is 1): those tie, and the lower index is chosen.
//
// One wave per token, no barriers: expert i 64 + lane is element i of a lane,
// so everything up to the choice is in registers.  The choice takes the
// largest c topk times.  c is held as an unsigned integer of the same order,
// split into two words: the largest high word is found with four DPP steps
// and four scalar maxima, and only experts that tie in it are compared in the
// low word.  Bound by latency, and for many tokens by vector issue (832
// instructions a token of 256 experts): one token of 256 experts 5.4 us, 4096
// tokens 10.3 us, of which 5.9 are issue (a workgroup per token that counted the
// better experts for each took 10.8 and 52 us).
#include "common.h"
#include "launch.h"
#include "route_groups.h"

namespace w8 {
namespace {

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));    // quad_perm [1,0,3,2]
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));    // quad_perm [2,3,0,1]
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));   // row_half_mirror
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false));   // row_ror:8
  return umax(umax((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16)),
              umax((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48)));
}

__device__ __forceinline__ double lane_double(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint64_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, lo | (hi << 32));
}

template <int CTRL>
__device__ __forceinline__ double dpp_double(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}

// NE: elements per lane (E <= 64 NE).  Dynamic LDS: c [E] and s [E], then
// (n_group > 1) the groups' scores [n_group].
template <int NE>
__global__ __launch_bounds__(64) void k_route_topk(RouteArgs a) {
  extern __shared__ __align__(16) double lds[];
  const int E = a.E, lane = threadIdx.x;
  const int64_t t = a.t0 + blockIdx.x;
  double* lc = lds;
  double* lw = lc + E;
  double* gs = lw + E;
  const double ninf = -__builtin_inf();

  float lf[NE], bias[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = i * 64 + lane;
    lf[i] = -__builtin_inff();
    bias[i] = 0.f;
    if (e < E) {
      if (a.dtype == 2) {
        lf[i] = static_cast<const float*>(a.logits)[t * E + e];
      } else {
        const uint32_t b = static_cast<const uint16_t*>(a.logits)[t * E + e];
        lf[i] = a.dtype == 1 ? h2f(b) : bf16_lo(b);
      }
      if (a.bias) bias[i] = a.bias[e];
    }
  }
  double s[NE];
  bool live[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    // a NaN compares false: masked, as -inf is; +inf is the largest finite
    live[i] = lf[i] > -__builtin_inff();
    lf[i] = live[i] ? fminf(lf[i], 3.40282347e38f) : -__builtin_inff();
  }
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < NE; ++i) s[i] = live[i] ? 1.0 / (1.0 + exp(-(double)lf[i])) : 0.0;
  } else {
    float mx = lf[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) mx = fmaxf(mx, lf[i]);
    mx = wave_max(mx);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      s[i] = live[i] ? exp((double)lf[i] - (double)mx) : 0.0;
      sum += s[i];
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
#pragma unroll
    for (int i = 0; i < NE; ++i) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
  }
  double c[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = i * 64 + lane;
    c[i] = live[i] ? (a.bias ? s[i] + (double)bias[i] : s[i]) : ninf;
    if (!(c[i] > ninf)) c[i] = ninf;   // a NaN bias masks its expert too
    if (e < E) {
      lc[e] = c[i];
      lw[e] = s[i];
    }
  }
  __syncthreads();   // one wave: orders its LDS accesses only
  if (a.n_group > 1) {
    // w lanes to a group take every w-th of its experts, then join
    const int per = a.per, w = 1 << a.lg_w, g = lane >> a.lg_w;
    double b1 = ninf, b2 = ninf;
    if (g < a.n_group)
      for (int j = lane & (w - 1); j < per; j += w) {
        const double v = lc[g * per + j];
        b2 = fmax(b2, fmin(b1, v));
        b1 = fmax(b1, v);
      }
    auto join = [&](double o1, double o2) {
      b2 = fmax(fmin(b1, o1), fmax(b2, o2));
      b1 = fmax(b1, o1);
    };
    // each step's partner holds the same as its neighbours that joined before
    if (w > 1) join(dpp_double<0xB1>(b1), dpp_double<0xB1>(b2));     // quad_perm [1,0,3,2]
    if (w > 2) join(dpp_double<0x4E>(b1), dpp_double<0x4E>(b2));     // quad_perm [2,3,0,1]
    if (w > 4) join(dpp_double<0x141>(b1), dpp_double<0x141>(b2));   // row_half_mirror
    if (w > 8) join(dpp_double<0x128>(b1), dpp_double<0x128>(b2));   // row_ror:8
    if (w > 16) join(__shfl_xor(b1, 16, 64), __shfl_xor(b2, 16, 64));
    if ((lane & (w - 1)) == 0 && g < a.n_group) gs[g] = a.group_top == 2 && b2 > ninf ? b1 + b2 : b1;
    __syncthreads();
    // lane g: the place of group g; a bit per group that stays
    const double v = lane < a.n_group ? gs[lane] : ninf;
    int place = 0;
    for (int j = 0; j < a.n_group; ++j) {
      const double o = lane_double(v, j);
      place += (int)(o > v) | ((int)(o == v) & (int)(j < lane));
    }
    const uint64_t stays = __ballot(lane < a.n_group && place < a.topk_group);
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = i * 64 + lane;
      if (!route_group_stays(stays, (uint32_t)e, (uint32_t)E, a.per_magic)) c[i] = ninf;
    }
  }

  // the same order as unsigned integers, 0 for an expert that cannot be chosen
  uint32_t hi[NE], lo[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    uint64_t b = __builtin_bit_cast(uint64_t, c[i] + 0.0);   // -0 becomes 0
    b = b >> 63 ? ~b : b | (1ull << 63);
    if (!(c[i] > ninf)) b = 0;
    hi[i] = (uint32_t)(b >> 32);
    lo[i] = (uint32_t)b;
  }
  int mine = -1;   // lane j: the j-th choice
  for (int j = 0; j < a.topk; ++j) {
    uint32_t v = hi[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) v = umax(v, hi[i]);
    const uint32_t m = wave_umax(v);
    if (m == 0) break;
    uint64_t at[NE];
    int n = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      at[i] = __ballot(hi[i] == m);
      n += __popcll(at[i]);
    }
    if (n > 1) {
      v = 0;
#pragma unroll
      for (int i = 0; i < NE; ++i) v = umax(v, hi[i] == m ? lo[i] : 0u);
      const uint32_t ml = wave_umax(v);
#pragma unroll
      for (int i = 0; i < NE; ++i) at[i] = __ballot(hi[i] == m && lo[i] == ml);
    }
    int e = 0;
#pragma unroll
    for (int i = NE - 1; i >= 0; --i)
      if (at[i]) e = i * 64 + __ffsll((unsigned long long)at[i]) - 1;
    if (lane == j) mine = e;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (i * 64 + lane == e) hi[i] = 0;
  }
  double w = mine >= 0 ? lw[mine] : 0.0;
  if (a.renormalise) {
    double sum = 0.0;
    for (int j = 0; j < a.topk; ++j) sum += lane_double(w, j);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  if (lane < a.topk) {
    a.ids[t * a.topk + lane] = mine;
    a.weights[t * a.topk + lane] = (float)(w * a.scale);
  }
}

template <int NE>
hipError_t route_launch(RouteArgs a, int64_t T, hipStream_t st) {
  const size_t lds = (size_t)a.E * 16 + (a.n_group > 1 ? (size_t)a.n_group * 8 : 0);
  constexpr int64_t kPart = int64_t(1) << 24;   // a launch holds fewer than 2^32 threads
  for (a.t0 = 0; a.t0 < T; a.t0 += kPart) {
    const int64_t n = T - a.t0 < kPart ? T - a.t0 : kPart;
    hipLaunchKernelGGL((k_route_topk<NE>), dim3((unsigned)n), dim3(64), lds, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_route_topk(RouteArgs a, int64_t T, hipStream_t st) {
  const int per = a.per = a.E / a.n_group;
  a.lg_w = 0;
  while ((2 << a.lg_w) * a.n_group <= 64) ++a.lg_w;
  a.per_magic = route_group_magic((uint32_t)per);
  if (a.E <= 64) return route_launch<1>(a, T, st);
  if (a.E <= 128) return route_launch<2>(a, T, st);
  if (a.E <= 256) return route_launch<4>(a, T, st);
  if (a.E <= 512) return route_launch<8>(a, T, st);
  return route_launch<16>(a, T, st);
}

}  // namespace w8
