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
// of exp and of the sum would decide between experts whose logits differ.
#include "common.h"
#include "launch.h"

namespace w8 {
namespace {

__device__ __forceinline__ double block_reduce(double v, bool mx, double* red, int nw) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const double o = __shfl_xor(v, d, 64);
    v = mx ? fmax(v, o) : v + o;
  }
  if (nw > 1) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
    for (int w = 1; w < nw; ++w) v = mx ? fmax(v, red[w]) : v + red[w];
  }
  return v;
}

// One workgroup per token, one expert per thread (blockDim.x >= E).  An
// expert's place in the order is the number of experts before it: larger c,
// or equal c and a lower index.  Places are distinct whatever the values
// (masked experts hold -inf), so each of the topk slots is written once.
__global__ __launch_bounds__(1024) void k_route_topk(RouteArgs a) {
  __shared__ double c[1024];
  __shared__ double top[1024][2];
  __shared__ double sel[64];
  __shared__ double red[2][16];
  __shared__ uint8_t stays[1024];
  const int64_t t = blockIdx.x;
  const int e = threadIdx.x;
  const int E = a.E, nw = blockDim.x >> 6;
  const bool in = e < E;
  const double ninf = -__builtin_inf();
  float lf = -__builtin_inff();
  if (in) {
    const int64_t i = t * E + e;
    if (a.dtype == 2) {
      lf = static_cast<const float*>(a.logits)[i];
    } else {
      const uint32_t b = static_cast<const uint16_t*>(a.logits)[i];
      lf = a.dtype == 1 ? h2f(b) : bf16_lo(b);
    }
  }
  // a NaN compares false: masked, as -inf is; +inf is the largest finite
  const bool live = lf > -__builtin_inff();
  const double l = live ? (double)fminf(lf, 3.40282347e38f) : ninf;
  double s;
  if (a.sigmoid) {
    s = live ? 1.0 / (1.0 + exp(-l)) : 0.0;
  } else {
    const double mx = block_reduce(l, true, red[0], nw);
    s = live ? exp(l - mx) : 0.0;
    const double sum = block_reduce(s, false, red[1], nw);
    s = sum > 0.0 ? s / sum : 0.0;
  }
  double ce = live ? (a.bias ? s + (double)a.bias[e] : s) : ninf;
  if (!(ce > ninf)) ce = ninf;   // a NaN bias masks its expert too
  if (in) c[e] = ce;
  __syncthreads();
  if (a.n_group > 1) {
    const int per = E / a.n_group;
    const int g = in ? e / per : 0;
    if (in) {
      int place = 0;
      for (int j = g * per; j < g * per + per; ++j) place += c[j] > ce || (c[j] == ce && j < e);
      if (place < 2) top[g][place] = ce;
    }
    __syncthreads();
    double* gs = &top[0][0];
    double score = 0.0;
    if (e < a.n_group) {
      score = top[e][0];
      if (a.group_top == 2 && per > 1 && top[e][1] > ninf) score += top[e][1];
    }
    __syncthreads();
    if (e < a.n_group) gs[e] = score;
    __syncthreads();
    if (e < a.n_group) {
      int place = 0;
      for (int j = 0; j < a.n_group; ++j) place += gs[j] > score || (gs[j] == score && j < e);
      stays[e] = place < a.topk_group;
    }
    __syncthreads();
    if (in && !stays[g]) c[e] = ce = ninf;
    __syncthreads();
  }
  int place = 1 << 30;
  if (in) {
    place = 0;
    for (int j = 0; j < E; ++j) place += c[j] > ce || (c[j] == ce && j < e);
  }
  const bool some = ce > ninf;
  if (place < a.topk) {
    a.ids[t * a.topk + place] = some ? e : -1;
    sel[place] = some ? s : 0.0;
  }
  __syncthreads();
  if (place < a.topk) {
    double w = some ? s : 0.0;
    if (a.renormalise) {
      double sum = 0.0;
      for (int j = 0; j < a.topk; ++j) sum += sel[j];
      w = sum > 0.0 ? w / sum : 0.0;
    }
    a.weights[t * a.topk + place] = (float)(w * a.scale);
  }
}

}  // namespace

hipError_t launch_route_topk(const RouteArgs& a, int64_t T, hipStream_t st) {
  const unsigned nt = (unsigned)((a.E + 63) / 64 * 64);
  hipLaunchKernelGGL(k_route_topk, dim3((unsigned)T), dim3(nt), 0, st, a);
  return hipGetLastError();
}

}  // namespace w8
