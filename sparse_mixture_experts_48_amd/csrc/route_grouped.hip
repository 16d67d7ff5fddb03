// The grouped router: scores of given logits, a bias that steers the choice,
// a choice limited to the best groups of experts, gates of the chosen; and the
// gradient of the gates.
//
//   s_e = 1 / (1 + e^-l_e)   or   e^(l_e - m) / sum_i e^(l_i - m)
//   c_e = s_e + b_e
//   group score = sum of the group's group_top largest c (1 or 2); the
//   top_groups best groups stay; the K largest c among their experts are the
//   choice, ties to the lower index; gate = scale s / sum of the chosen s
//   (renormalised) or scale s.
//
// The choice is defined on float64 scores, so no rounding of float32 decides
// it.
//
// Simple form: one wave per token, lane l holds experts 64 i + l.
#include "common.h"
#include "fp8.h"

namespace moe {

namespace {

constexpr int kRT = 4;  // tokens (waves) per block

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmax(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

template <typename T> struct Lowest;
template <> struct Lowest<float> { static constexpr float v = -3.402823466e+38f; };
template <> struct Lowest<bf16_t> { static constexpr float v = -3.38953139e+38f; };

// scores of the lane's experts (0 where masked); false in ok where an expert cannot be chosen
template <typename T>
__device__ __forceinline__ void scores64(const T* row, int E, bool sigmoid, int lane, double* s, bool* ok) {
  double l[8];
  double m = -INFINITY;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = 64 * i + lane;
    s[i] = 0.0;
    ok[i] = false;
    l[i] = -INFINITY;
    if (e < E) {
      const float v = Elem<T>::load(row + e);
      ok[i] = !(v <= Lowest<T>::v);
      if (ok[i]) l[i] = v;
    }
    m = (l[i] > m || l[i] != l[i]) ? l[i] : m;
  }
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (ok[i]) s[i] = 1.0 / (1.0 + exp(-l[i]));
      if (s[i] != s[i]) s[i] = 0.0, ok[i] = false;
    }
    return;
  }
  m = wave_max(m);
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (ok[i]) s[i] = exp(l[i] - m);
    sum += s[i];
  }
  sum = wave_sum(sum);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (ok[i]) s[i] = s[i] / sum;
    if (s[i] != s[i]) s[i] = 0.0, ok[i] = false;
  }
}

template <typename T>
__global__ __launch_bounds__(64 * kRT) void route_grouped_kernel(GroupedRouteArgs a, int32_t* __restrict__ topk_idx,
                                                                 float* __restrict__ topk_gate) {
  const int lane = threadIdx.x % 64, w = threadIdx.x / 64;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRT + w;
  __shared__ double gsc[kRT][kMaxGroups];
  const bool live = t < a.T;
  double s[8], c[8];
  bool ok[8];
  const int gs = a.E / a.groups;
  if (live) {
    scores64(static_cast<const T*>(a.logits) + t * a.E, a.E, a.sigmoid, lane, s, ok);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      c[i] = ok[i] ? s[i] + (a.bias != nullptr ? static_cast<double>(a.bias[64 * i + lane]) : 0.0) : -INFINITY;
  }
  if (a.top_groups < a.groups) {
    if (live) {
      for (int g = 0; g < a.groups; ++g) {
        double b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = 64 * i + lane;
          if (e / gs != g) continue;
          if (c[i] > b1) { b2 = b1; b1 = c[i]; }
          else if (c[i] > b2) b2 = c[i];
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
          const double o1 = __shfl_xor(b1, o), o2 = __shfl_xor(b2, o);
          const double lo = fmin(b1, o1);
          b1 = fmax(b1, o1);
          b2 = fmax(lo, fmax(b2, o2));
        }
        if (lane == 0) gsc[w][g] = a.group_top == 2 && b2 > -INFINITY ? b1 + b2 : b1;
      }
    }
    __syncthreads();
    if (live) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = 64 * i + lane;
        if (e >= a.E) continue;
        const int g = e / gs;
        const double v = gsc[w][g];
        int better = 0;
        for (int h = 0; h < a.groups; ++h) better += gsc[w][h] > v || (gsc[w][h] == v && h < g);
        if (better >= a.top_groups) c[i] = -INFINITY;
      }
    }
  }
  if (!live) return;
  double sel = 0.0, sum = 0.0;
  int id = kNoExpert;
  for (int j = 0; j < a.K; ++j) {
    double b = -INFINITY;
    int e = kNoExpert;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c[i] > b) { b = c[i]; e = 64 * i + lane; }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const double ob = __shfl_xor(b, o);
      const int oe = __shfl_xor(e, o);
      if (ob > b || (ob == b && oe < e)) { b = ob; e = oe; }
    }
    double sv = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (64 * i + lane == e) { sv = s[i]; c[i] = -INFINITY; }
    sv = wave_sum(sv);
    sum += sv;
    if (lane == j) { sel = sv; id = e; }
  }
  if (lane < a.K) {
    const double g = a.renorm ? sel / fmax(sum, 0x1p-126) : sel;
    topk_idx[t * a.K + lane] = id;
    topk_gate[t * a.K + lane] = static_cast<float>(static_cast<double>(a.scale) * g);
  }
}

template <typename T>
__global__ __launch_bounds__(64 * kRT) void route_grouped_bwd_kernel(GroupedRouteArgs a,
                                                                     const int32_t* __restrict__ topk_idx,
                                                                     const float* __restrict__ dgate,
                                                                     T* __restrict__ dlogits) {
  const int lane = threadIdx.x % 64, w = threadIdx.x / 64;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRT + w;
  if (t >= a.T) return;
  double s[8], d[8];
  bool ok[8];
  scores64(static_cast<const T*>(a.logits) + t * a.E, a.E, a.sigmoid, lane, s, ok);
  // sums over the chosen: of s, and of scale dgate s
  double D = 0.0, us = 0.0;
  for (int j = 0; j < a.K; ++j) {
    const int id = topk_idx[t * a.K + j];
    const double u = static_cast<double>(a.scale) * dgate[t * a.K + j];
    double sv = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (64 * i + lane == id) sv = s[i];
    sv = wave_sum(sv);
    D += sv;
    us += u * sv;
  }
  D = fmax(D, 0x1p-126);
#pragma unroll
  for (int i = 0; i < 8; ++i) d[i] = 0.0;
  for (int j = 0; j < a.K; ++j) {
    const int id = topk_idx[t * a.K + j];
    const double u = static_cast<double>(a.scale) * dgate[t * a.K + j];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (64 * i + lane == id) d[i] += a.renorm ? (u - us / D) / D : u;
  }
  double dot = 0.0;
  if (!a.sigmoid) {
#pragma unroll
    for (int i = 0; i < 8; ++i) dot += d[i] * s[i];
    dot = wave_sum(dot);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = 64 * i + lane;
    if (e >= a.E) continue;
    const double v = a.sigmoid ? d[i] * s[i] * (1.0 - s[i]) : s[i] * (d[i] - dot);
    Elem<T>::store(dlogits + t * a.E + e, static_cast<float>(v));
  }
}

}  // namespace

hipError_t launch_route_grouped(const GroupedRouteArgs& a, int32_t* topk_idx, float* topk_gate, hipStream_t st) {
  const dim3 grid((a.T + kRT - 1) / kRT), block(64 * kRT);
  if (a.bf16) hipLaunchKernelGGL(route_grouped_kernel<bf16_t>, grid, block, 0, st, a, topk_idx, topk_gate);
  else hipLaunchKernelGGL(route_grouped_kernel<float>, grid, block, 0, st, a, topk_idx, topk_gate);
  return hipGetLastError();
}

hipError_t launch_route_grouped_backward(const GroupedRouteArgs& a, const int32_t* topk_idx, const float* dgate,
                                         void* dlogits, hipStream_t st) {
  const dim3 grid((a.T + kRT - 1) / kRT), block(64 * kRT);
  if (a.bf16)
    hipLaunchKernelGGL(route_grouped_bwd_kernel<bf16_t>, grid, block, 0, st, a, topk_idx, dgate,
                       static_cast<bf16_t*>(dlogits));
  else
    hipLaunchKernelGGL(route_grouped_bwd_kernel<float>, grid, block, 0, st, a, topk_idx, dgate,
                       static_cast<float*>(dlogits));
  return hipGetLastError();
}

}  // namespace moe
