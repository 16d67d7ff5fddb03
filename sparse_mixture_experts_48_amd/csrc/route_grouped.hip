// The grouped router: scores of given logits, a bias that steers the choice,
// a choice limited to the best groups of experts, gates of the chosen; and the
// gradient of the gates.
//
//   s_e = 1 / (1 + e^-l_e)   or   e^(l_e - m) / sum_i e^(l_i - m)
//   c_e = s_e + b_e
//   group score = sum of the group's group_top largest c (1 or 2); the
//   top_groups best groups stay; the K largest c among their experts are the
//   choice, ties to the lower index; gate = scale s / sum of the chosen s
//   (renormalised; for softmax the softmax of the chosen logits) or scale s.
//
// The choice is defined on float64 scores, so no rounding of float32 decides
// it. It is made in float32 first: every comparison that matters (the kept
// groups against the others, each chosen expert against the next) is checked
// to be further apart than float32 can be wrong, and a wave that holds a token
// with a closer one makes its choice again in float64. Without a bias the
// scores rise with the logits, so the float32 pass compares the logits
// themselves, exactly: equal logits are equal scores, and only distances that
// float64 scores cannot tell apart (far out, where they saturate) go again.
//
// Layout: 16 lanes per token, four tokens per wave, one wave per block. Lane l
// of a token holds experts 64 i + 4 l .. + 3 (16-byte loads), Q = ceil(E / 64)
// such runs. Maxima over a token are four row rotations folded into v_max /
// v_min (DPP), so a pick costs about six vector instructions per expert of the
// lane, and the group scores go through LDS (one lane per group scans it).
// Bound: instruction issue for large batches (the rows are read once), the
// latency of one wave for small ones.
#include <type_traits>

#include "common.h"
#include "fp8.h"

namespace moe {

namespace {

constexpr int kLanes = 16;            // lanes per token
constexpr int kTok = 64 / kLanes;     // tokens per wave
constexpr float kNone = -__builtin_huge_valf();  // the key of an expert that cannot be chosen

// lane l gets the value of lane (l + N) % 16 of its row of 16
template <int N>
__device__ __forceinline__ int row_ror(int v) { return __builtin_amdgcn_update_dpp(v, v, 0x120 + N, 0xF, 0xF, false); }
template <int N>
__device__ __forceinline__ float row_ror(float v) { return __int_as_float(row_ror<N>(__float_as_int(v))); }
template <int N>
__device__ __forceinline__ double row_ror(double v) {
  return __hiloint2double(row_ror<N>(__double2hiint(v)), row_ror<N>(__double2loint(v)));
}
__device__ __forceinline__ float vmax(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double vmax(double a, double b) { return fmax(a, b); }
template <typename V>
__device__ __forceinline__ V row_max(V v) {
  v = vmax(v, row_ror<8>(v));
  v = vmax(v, row_ror<4>(v));
  v = vmax(v, row_ror<2>(v));
  return vmax(v, row_ror<1>(v));
}
template <typename V>
__device__ __forceinline__ V row_sum(V v) {
  v += row_ror<8>(v);
  v += row_ror<4>(v);
  v += row_ror<2>(v);
  return v + row_ror<1>(v);
}
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
  v = min(v, static_cast<uint32_t>(row_ror<8>(static_cast<int>(v))));
  v = min(v, static_cast<uint32_t>(row_ror<4>(static_cast<int>(v))));
  v = min(v, static_cast<uint32_t>(row_ror<2>(static_cast<int>(v))));
  return min(v, static_cast<uint32_t>(row_ror<1>(static_cast<int>(v))));
}

// Orders the LDS accesses of a wave's lanes (the hardware runs a wave's LDS
// instructions in order; this keeps the compiler to it).
__device__ __forceinline__ void wave_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

template <typename T> struct Lowest;
template <> struct Lowest<float> { static constexpr float v = -3.402823466e+38f; };
template <> struct Lowest<bf16_t> { static constexpr float v = -3.38953139e+38f; };

// Logits of the lane's experts; -infinity where masked or past the last one.
template <typename T, int Q>
__device__ __forceinline__ void load_logits(const T* row, int E, int l, bool live, float* v) {
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int e = 64 * i + 4 * l;
    if (E % 4 == 0) {  // rows start on a multiple of four values
      if (live && e < E) {
        if constexpr (sizeof(T) == 4) {
          const f32x4_t x = *reinterpret_cast<const f32x4_t*>(row + e);
#pragma unroll
          for (int c = 0; c < 4; ++c) v[4 * i + c] = x[c];
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(row + e);
          v[4 * i] = __uint_as_float(x.x << 16);
          v[4 * i + 1] = __uint_as_float(x.x & 0xFFFF0000u);
          v[4 * i + 2] = __uint_as_float(x.y << 16);
          v[4 * i + 3] = __uint_as_float(x.y & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) v[4 * i + c] = kNone;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) v[4 * i + c] = live && e + c < E ? Elem<T>::load(row + e + c) : kNone;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) v[4 * i + c] = v[4 * i + c] <= Lowest<T>::v ? kNone : v[4 * i + c];
  }
}

__device__ __forceinline__ float exp_(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }
__device__ __forceinline__ double exp_(double x) { return exp(x); }
__device__ __forceinline__ float rcp_(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ double rcp_(double x) { return 1.0 / x; }

// Row maximum and sum of e^(l - m) (m = 0 for a row with nothing left; a NaN or
// +infinity makes the sum NaN).
template <typename V, int N>
__device__ __forceinline__ void row_softmax(const float* l, V* m, V* sum) {
  float mm = kNone;
#pragma unroll
  for (int i = 0; i < N; ++i) mm = fmaxf(mm, l[i]);
  mm = row_max(mm);
  *m = mm == kNone ? V(0) : V(mm);
  V s = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) s += exp_(V(l[i]) - *m);
  *sum = row_sum(s);
}

// Whether a (the larger) and b may be in another order, or equal, in float64.
// exact: both are logits themselves, whose distinct values can have equal
// scores within 1e-8 of each other, above `high` (1 / (1 + e^-l) near 1) and
// below `low` (e^l underflows).
__device__ __forceinline__ bool unsure(float a, float b, bool exact, float low, float high, float err) {
  if (b == kNone) return false;
  const float gap = a - b;
  if (exact) return gap > 0.0f && (gap < 1e-8f || a > high || b < low);
  return !(gap > err * (1.0f + fabsf(a)));
}

// The choice of one token by its 16 lanes in V = float or double. id: lane j's
// j-th choice (kNoExpert: none left). Returns whether float could not be sure.
template <typename V, int Q>
__device__ bool choose(const GroupedRouteArgs& a, const float* l, const int lane, V* lds, V* lds_g, int* id) {
  constexpr int N = 4 * Q;
  constexpr bool F = sizeof(V) == 4;
  // float: the scores' own error (a few steps of 2^-24 of a value up to 1), twice, with room; relative to the sum with
  // the bias, whose rounding is relative to it
  constexpr float kErr = 0x1p-20f;
  const V none = -__builtin_huge_val();
  V key[N];
  float far = -700.0f, near = a.sigmoid ? 20.0f : -kNone;
  bool poisoned = false;
  V m = 0, sum = 0;
  const bool softmax = !a.sigmoid;
  const bool exact = F && a.bias == nullptr;               // keys are the logits themselves
  const bool group_exact = exact && a.group_top == 1;      // and so are group scores
  const bool grouped = a.top_groups < a.groups;
  const bool need_s = !exact || (grouped && !group_exact);
  if (softmax) {
    row_softmax<V, N>(l, &m, &sum);
    poisoned = sum != sum;
    far = static_cast<float>(m) - 700.0f;
    sum = rcp_(sum);
  }
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    f32x4_t bias = {0.f, 0.f, 0.f, 0.f};
    if (a.bias != nullptr) {
      const int e = 64 * i + 4 * lane;
      if (a.E % 4 == 0) bias = *reinterpret_cast<const f32x4_t*>(a.bias + min(e, a.E - 4));
      else
#pragma unroll
        for (int c = 0; c < 4; ++c) bias[c] = a.bias[min(e + c, a.E - 1)];
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int e = 64 * i + 4 * lane + c;
      const float x = l[4 * i + c];
      const bool ok = x > kNone && !poisoned;  // (a NaN is not larger)
      V s = 0;
      if (need_s) s = (softmax ? exp_(V(x) - m) * sum : rcp_(V(1) + exp_(-V(x)))) + V(bias[c]);
      key[4 * i + c] = ok ? (exact ? V(x) : s) : none;
      if (grouped && e < a.E) lds[e] = ok ? (group_exact ? V(x) : s) : none;
    }
  }
  bool close = false;
  if (grouped) {
    wave_order();
    const int gs = a.E / a.groups;
    // scores of groups lane and lane + 16: the two largest of each, scanned from a start of the lane's own
    V score[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int g = lane + 16 * h;
      V b1 = none, b2 = none;
      if (g < a.groups) {
        int at = 4 * g % gs;
        for (int k = 0; k < gs; ++k) {
          const V v = lds[g * gs + at];
          b2 = vmax(b2, v < b1 ? v : b1);
          b1 = vmax(b1, v);
          at = at + 1 == gs ? 0 : at + 1;
        }
        lds_g[g] = score[h] = a.group_top == 2 && b2 > none ? b1 + b2 : b1;
      } else {
        score[h] = none;
      }
    }
    wave_order();
    uint32_t kept = 0;
    V low = -none, high = none;  // the worst kept score, the best other one
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int g = lane + 16 * h;
      int better = 0;
      for (int o = 0; o < a.groups; ++o) {
        const V v = lds_g[o];
        better += v > score[h] || (v == score[h] && o < g);
      }
      const bool keep = g < a.groups && better < a.top_groups;
      if (keep) low = low < score[h] ? low : score[h];
      else high = vmax(high, score[h]);
      kept |= static_cast<uint32_t>(__ballot(keep) >> (threadIdx.x / kLanes * kLanes) & 0xFFFF) << (16 * h);
    }
    if constexpr (F) {
      low = -row_max(-low);
      high = row_max(high);
      close = unsure(low, high, group_exact, far, near, 2.0f * kErr);
    }
    const uint32_t magic = ((1u << 20) + gs - 1) / gs;  // e / gs for e < 512
#pragma unroll
    for (int i = 0; i < Q; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t e = 64 * i + 4 * lane + c;
        if (!(kept >> ((e * magic) >> 20) & 1)) key[4 * i + c] = none;
      }
  }
  V last = -none;
  *id = kNoExpert;
  for (int j = 0; j <= (F ? a.K : a.K - 1); ++j) {  // float: one more, to compare the last with
    V b = none;
#pragma unroll
    for (int i = 0; i < N; ++i) b = vmax(b, key[i]);
    b = row_max(b);
    if constexpr (F) close |= j > 0 && unsure(last, b, exact, far, near, kErr);
    last = b;
    uint32_t e = kNoExpert;
#pragma unroll
    for (int i = N - 1; i >= 0; --i) e = key[i] == b ? 64 * (i / 4) + 4 * lane + i % 4 : e;
    e = row_min(b > none ? e : kNoExpert);
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = e == 64 * (i / 4) + 4 * lane + i % 4 ? none : key[i];
    if (lane == j) *id = static_cast<int>(e);
  }
  if (lane >= a.K) *id = kNoExpert;
  return close;
}

template <typename T, int Q>
__global__ __launch_bounds__(64) void route_grouped_kernel(GroupedRouteArgs a, int32_t* __restrict__ topk_idx,
                                                           float* __restrict__ topk_gate) {
  __shared__ float lds32[kTok][64 * Q];
  __shared__ float lds32g[kTok][kMaxGroups];
  const int lane = threadIdx.x % kLanes, tok = threadIdx.x / kLanes;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kTok + tok;
  const bool live = t < a.T;
  const T* row = static_cast<const T*>(a.logits) + t * a.E;
  float l[4 * Q];
  load_logits<T, Q>(row, a.E, lane, live, l);
  int id;
  const bool close = choose<float, Q>(a, l, lane, lds32[tok], lds32g[tok], &id);
  if (__ballot(close) != 0) {
    __shared__ double lds64[kTok][64 * Q];
    __shared__ double lds64g[kTok][kMaxGroups];
    choose<double, Q>(a, l, lane, lds64[tok], lds64g[tok], &id);
  }
  // gates in float64 (one exponential per chosen expert)
  const bool got = id != kNoExpert;
  const double x = got && live ? static_cast<double>(Elem<T>::load(row + id)) : 0.0;
  double s = 0.0, D = 1.0;
  if (a.sigmoid) {
    s = got ? 1.0 / (1.0 + exp(-x)) : 0.0;
    if (a.renorm) D = fmax(row_sum(s), 0x1p-126);
  } else {
    float m, sum;
    if (a.renorm) {
      m = row_max(got ? static_cast<float>(x) : kNone);
      s = got ? exp(x - static_cast<double>(m)) : 0.0;
      D = row_sum(s);
    } else {
      row_softmax<float, 4 * Q>(l, &m, &sum);
      s = got ? exp(x - static_cast<double>(m)) : 0.0;
      D = sum;
    }
  }
  if (live && lane < a.K) {
    topk_idx[t * a.K + lane] = id;
    topk_gate[t * a.K + lane] = got ? static_cast<float>(static_cast<double>(a.scale) * s / D) : 0.0f;
  }
}

// Gradient. With u = scale dgate, over the chosen:
//   renormalised sigmoid: ds_j = (u_j - sum_k u_k s_k / D) / D, D = sum_k s_k;  dl_j = ds_j s_j (1 - s_j)
//   renormalised softmax: g = softmax of the chosen logits;  dl_j = g_j (u_j - sum_k g_k u_k)
//   raw sigmoid: dl_j = u_j s_j (1 - s_j)
//   raw softmax: dl_e = p_e (u_e - sum_k u_k p_k) for every expert (u_e = 0 where not chosen)
// The K values of a token are formed in float64 by K of its lanes (the same id
// twice adds up); a row is zeroed in LDS, the values dropped in and the row
// stored in runs of four. Only raw softmax reads the whole row of logits.
// Bound: the writes (T E values) for large batches.
template <typename T, int Q>
__global__ __launch_bounds__(64) void route_grouped_bwd_kernel(GroupedRouteArgs a, const int32_t* __restrict__ topk_idx,
                                                               const float* __restrict__ dgate,
                                                               T* __restrict__ dlogits) {
  __shared__ f32x4_t rows[kTok][16 * Q];
  const int lane = threadIdx.x % kLanes, tok = threadIdx.x / kLanes;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kTok + tok;
  const bool live = t < a.T;
  const T* row = static_cast<const T*>(a.logits) + t * a.E;
  const bool mine = live && lane < a.K;
  int id = mine ? topk_idx[t * a.K + lane] : kNoExpert;
  const double u = mine ? static_cast<double>(a.scale) * dgate[t * a.K + lane] : 0.0;
  bool got = id >= 0 && id < a.E;
  const float xl = got ? Elem<T>::load(row + id) : 0.0f;
  got = got && xl > Lowest<T>::v;  // a masked expert's score is 0, and so is its gradient; NaN likewise
  const double x = got ? static_cast<double>(xl) : 0.0;
  const bool full = !a.sigmoid && !a.renorm;
  float l[4 * Q];
  double v = 0.0;
  float m = 0.0f, sum = 1.0f, dot = 0.0f;
  if (a.sigmoid) {
    const double s = got ? 1.0 / (1.0 + exp(-x)) : 0.0;
    double ds = u;
    if (a.renorm) {
      const double D = fmax(row_sum(s), 0x1p-126), us = row_sum(got ? u * s : 0.0);
      ds = (u - us / D) / D;
    }
    v = ds * s * (1.0 / (1.0 + exp(x)));  // 1 - s without its cancellation
  } else if (a.renorm) {
    const double top = static_cast<double>(row_max(got ? static_cast<float>(x) : kNone));
    const double ex = got ? exp(x - top) : 0.0;
    const double D = row_sum(ex);
    const double gj = D > 0.0 ? ex / D : 0.0;
    v = gj * (u - row_sum(got ? gj * u : 0.0));
  } else {
    load_logits<T, Q>(row, a.E, lane, live, l);
    row_softmax<float, 4 * Q>(l, &m, &sum);
    if (sum != sum || sum == 0.0f) got = false, sum = 1.0f, m = -kNone;  // every score is 0 (or NaN): no gradient
    sum = 1.0f / sum;
    const double p = got ? exp(x - static_cast<double>(m)) * static_cast<double>(sum) : 0.0;
    v = got ? p * u : 0.0;
    dot = static_cast<float>(row_sum(v));
  }
  v = got ? v : 0.0;
  id = got ? id : kNoExpert;
  // the same id in several choices: each of their lanes takes the sum, in choice order
  double total = 0.0;
  for (int k = 0; k < a.K; ++k) {
    const double vk = __shfl(v, (threadIdx.x & 48) + k);
    const int ik = __shfl(id, (threadIdx.x & 48) + k);
    total += ik == id ? vk : 0.0;
  }
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    f32x4_t z = {0.f, 0.f, 0.f, 0.f};
    if (full) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float xx = l[4 * i + c];
        z[c] = xx > kNone && m < -kNone ? -(exp_(xx - m) * sum) * dot : 0.0f;
      }
    }
    rows[tok][16 * i + lane] = z;
  }
  wave_order();
  float* const r = reinterpret_cast<float*>(rows[tok]);
  if (id != kNoExpert) r[id] = full ? static_cast<float>(total + static_cast<double>(r[id])) : static_cast<float>(total);
  wave_order();
  if (!live) return;
  T* const out = dlogits + t * a.E;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int e = 64 * i + 4 * lane;
    if (e >= a.E) continue;
    const f32x4_t z = rows[tok][16 * i + lane];
    if (a.E % 4 == 0) {
      if constexpr (sizeof(T) == 4) *reinterpret_cast<f32x4_t*>(out + e) = z;
      else *reinterpret_cast<uint2*>(out + e) = make_uint2(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]));
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (e + c < a.E) Elem<T>::store(out + e + c, z[c]);
    }
  }
}

// Q = ceil(E / 64), up to 8; 5 and 7 run as 6 and 8
template <typename T, typename F>
hipError_t by_width(int E, F&& f) {
  switch ((E + 63) / 64) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 3: return f(std::integral_constant<int, 3>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 5:
    case 6: return f(std::integral_constant<int, 6>{});
    default: return f(std::integral_constant<int, 8>{});
  }
}

}  // namespace

hipError_t launch_route_grouped(const GroupedRouteArgs& a, int32_t* topk_idx, float* topk_gate, hipStream_t st) {
  const dim3 grid((a.T + kTok - 1) / kTok), block(64);
  auto run = [&](auto elem) {
    using T = decltype(elem);
    return by_width<T>(a.E, [&](auto q) {
      hipLaunchKernelGGL((route_grouped_kernel<T, decltype(q)::value>), grid, block, 0, st, a, topk_idx, topk_gate);
      return hipGetLastError();
    });
  };
  return a.bf16 ? run(bf16_t{}) : run(float{});
}

hipError_t launch_route_grouped_backward(const GroupedRouteArgs& a, const int32_t* topk_idx, const float* dgate,
                                         void* dlogits, hipStream_t st) {
  const dim3 grid((a.T + kTok - 1) / kTok), block(64);
  auto run = [&](auto elem) {
    using T = decltype(elem);
    return by_width<T>(a.E, [&](auto q) {
      hipLaunchKernelGGL((route_grouped_bwd_kernel<T, decltype(q)::value>), grid, block, 0, st, a, topk_idx, dgate,
                         static_cast<T*>(dlogits));
      return hipGetLastError();
    });
  };
  return a.bf16 ? run(bf16_t{}) : run(float{});
}

}  // namespace moe
