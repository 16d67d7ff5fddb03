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
// it. It is made in float32 first, and every comparison that matters (the kept
// groups against the others, each chosen expert against the next) is checked
// to be further apart than float32 can be wrong. Without a bias the scores rise
// with the logits, so the float32 pass compares the logits themselves, exactly.
// Where chosen scores are too close (sigmoid: about one token in 2000 of 256
// experts), the K + 1 best are ordered again by float64 scores, one lane each;
// for the rest (groups too close, saturated logits) the wave makes that token's
// choice again, in float64 throughout.
//
// Layout: LPT = 16 lanes per token (four tokens per wave) for large batches, 64
// for small ones; one wave per block. Lane l of a token holds experts
// 4 LPT i + 4 l .. + 3 (16-byte loads). Maxima over a token are row rotations
// folded into v_max / v_min (DPP) and, over 64 lanes, two half swaps, so a pick
// costs about six vector instructions per expert of the lane; the group scores
// go through LDS, one lane per group reading it eight values at a time.
// Bound: instruction issue for large batches (the rows are read once), the
// latency of one wave for small ones. Measured: 256 experts in 8 groups, K = 8,
// 8192 tokens 13 us (0.7 TB/s), 16 tokens 7 us.
#include <type_traits>

#include "common.h"
#include "fp8.h"

namespace moe {

namespace {

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
// The other half of 32 (or 16) lanes' value beside each lane's own: with both
// operands v, the swap leaves one half's values in every lane of r[0], the other's in r[1].
typedef unsigned u32_pair __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u32_pair swap32(unsigned v) { return __builtin_amdgcn_permlane32_swap(v, v, false, false); }
__device__ __forceinline__ u32_pair swap16(unsigned v) { return __builtin_amdgcn_permlane16_swap(v, v, false, false); }
template <typename V, typename F>
__device__ __forceinline__ V across_rows(V v, F&& op) {  // over the four rows of 16
  if constexpr (sizeof(V) == 4) {
    u32_pair r = swap16(__builtin_bit_cast(unsigned, v));
    v = op(__builtin_bit_cast(V, static_cast<unsigned>(r[0])), __builtin_bit_cast(V, static_cast<unsigned>(r[1])));
    r = swap32(__builtin_bit_cast(unsigned, v));
    return op(__builtin_bit_cast(V, static_cast<unsigned>(r[0])), __builtin_bit_cast(V, static_cast<unsigned>(r[1])));
  } else {
    u32_pair lo = swap16(__double2loint(v)), hi = swap16(__double2hiint(v));
    v = op(__hiloint2double(hi[0], lo[0]), __hiloint2double(hi[1], lo[1]));
    lo = swap32(__double2loint(v)), hi = swap32(__double2hiint(v));
    return op(__hiloint2double(hi[0], lo[0]), __hiloint2double(hi[1], lo[1]));
  }
}
template <int LPT, typename V, typename F>
__device__ __forceinline__ V reduce(V v, F&& op) {
  v = op(v, row_ror<8>(v));
  v = op(v, row_ror<4>(v));
  v = op(v, row_ror<2>(v));
  v = op(v, row_ror<1>(v));
  if constexpr (LPT == 64) v = across_rows(v, op);
  return v;
}
template <int LPT, typename V>
__device__ __forceinline__ V row_max(V v) {
  return reduce<LPT>(v, [](V a, V b) { return vmax(a, b); });
}
template <int LPT, typename V>
__device__ __forceinline__ V row_sum(V v) {
  return reduce<LPT>(v, [](V a, V b) { return a + b; });
}
template <int LPT>
__device__ __forceinline__ int row_min(int v) {
  return reduce<LPT>(v, [](int a, int b) { return min(a, b); });
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
template <int LPT, int Q, typename T>
__device__ __forceinline__ void load_logits(const T* row, int E, int l, bool live, float* v) {
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int e = 4 * LPT * i + 4 * l;
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
// +infinity makes the sum NaN). The lane's terms are added in pairs: at most 11
// roundings from a term to the sum.
template <int LPT, typename V, int N>
__device__ __forceinline__ void row_softmax(const float* l, V* m, V* sum) {
  float mm = kNone;
#pragma unroll
  for (int i = 0; i < N; ++i) mm = fmaxf(mm, l[i]);
  mm = row_max<LPT>(mm);
  *m = mm == kNone ? V(0) : V(mm);
  V s[N];
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = exp_(V(l[i]) - *m);
#pragma unroll
  for (int w = 1; w < N; w *= 2)
#pragma unroll
    for (int i = 0; i + w < N; i += 2 * w) s[i] += s[i + w];
  *sum = row_sum<LPT>(s[0]);
}

// What the float32 pass found of a token's choice.
enum { SURE = 0, REORDER = 1, AGAIN = 2 };

// Whether float64 may order a and b (a >= b in float32) otherwise, or find them
// equal. exact: both are logits themselves, whose distinct values can have
// equal scores within 1e-8 of each other, above `high` (1 / (1 + e^-l) near 1) and
// below `low` (e^l underflows). Else both are off by at most err / 2.
__device__ __forceinline__ bool unsure(float a, float b, bool exact, float low, float high, float err) {
  if (b == kNone) return false;
  const float gap = a - b;
  if (exact) return gap > 0.0f && (gap < 1e-8f || a > high || b < low);
  return !(gap > err);
}

// The choice of one token by its LPT lanes in V = float or double. id: lane j's
// j-th choice (kNoExpert: none left), lane K's the next one after them (float
// only). Returns what float was not sure of.
// lds: E + groups values, group g's from g (E / groups + 1) on (one value of
// padding each, so that the lanes that scan them meet in different banks).
template <int LPT, int Q, typename V>
__device__ int choose(const GroupedRouteArgs& a, const float* l, const int lane, V* lds, V* lds_g, int* id) {
  constexpr int N = 4 * Q;
  constexpr bool F = sizeof(V) == 4;
  // float: two values c are off by at most err + kRound |c| together. c = s + b rounds by 2^-24 |c|, each of two (with
  // room: 2^-21). A sigmoid score is off by s (1 - s) (|l| 2^-23 + 2^-23) from the exponential and 1.5 2^-23 from the sum
  // and the reciprocal: together below 2^-22.2, two of them below 2^-21. A softmax score p by p |l - m| 2^-23 <= 0.37
  // 2^-23 p_max from its exponent, 3 2^-23 p from its roundings, and by the sum, shared by all of the row: 11 roundings
  // of 2^-24, 2^-23 sum p |l - m| <= ln(512) 2^-23, 2^-23 for the reciprocal; two of them below 2^-18 p_max.
  constexpr float kRound = 0x1p-21f;
  float err = 0x1p-21f;
  const V none = -__builtin_huge_val();
  const bool softmax = !a.sigmoid;
  const bool exact = F && a.bias == nullptr;           // keys are the logits themselves
  const bool group_exact = exact && a.group_top == 1;  // and so are group scores
  const bool grouped = a.top_groups < a.groups;
  float far = -700.0f, near = a.sigmoid ? 20.0f : -kNone;
  bool poisoned = false;
  V m = 0, sum = 0;
  if (softmax) {
    row_softmax<LPT, V, N>(l, &m, &sum);
    poisoned = sum != sum;
    far = static_cast<float>(m) - 700.0f;
    if constexpr (F) err = 0x1p-18f * rcp_(sum);
  }
  V key[N];
  if (!exact || (grouped && !group_exact)) {
    if (softmax) {
      const V inv = rcp_(sum);
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = exp_(V(l[i]) - m) * inv;
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = rcp_(V(1) + exp_(-V(l[i])));
    }
    if (a.bias != nullptr) {
      float bias[N];
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const int e = 4 * LPT * i + 4 * lane;
        if (a.E % 4 == 0) {
          const f32x4_t b = *reinterpret_cast<const f32x4_t*>(a.bias + min(e, a.E - 4));
#pragma unroll
          for (int c = 0; c < 4; ++c) bias[4 * i + c] = b[c];
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) bias[4 * i + c] = a.bias[min(e + c, a.E - 1)];
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] += V(bias[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = V(l[i]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) key[i] = l[i] > kNone && !poisoned ? key[i] : none;  // (a NaN is not larger)
  int found = SURE;
  if (grouped) {
    const int gs = a.E / a.groups;
    const uint32_t magic = ((1u << 20) + gs - 1) / gs;  // e / gs for e < 2048: e (magic gs - 2^20) < 2^20
    uint32_t grp[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t e = 4 * LPT * (i / 4) + 4 * lane + i % 4;
      grp[i] = (e * magic) >> 20;
      if (e < static_cast<uint32_t>(a.E)) lds[e + grp[i]] = key[i];
    }
    if (exact && !group_exact) {  // the choice itself is on the logits
#pragma unroll
      for (int i = 0; i < N; ++i) key[i] = l[i] > kNone && !poisoned ? V(l[i]) : none;
    }
    wave_order();
    constexpr int H = LPT == 64 ? 1 : kMaxGroups / LPT;  // groups lane, lane + LPT
    V score[H], size = 0;  // size: the largest sum of magnitudes a score is formed from
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int g = lane + LPT * h;
      V b1 = none, b2 = none;
      const V* const mine = lds + min(g, a.groups - 1) * (gs + 1);
      for (int k = 0; k < gs; k += 8) {
        V v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = mine[min(k + u, gs - 1)];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const V x = k + u < gs ? v[u] : none;
          b2 = vmax(b2, x < b1 ? x : b1);
          b1 = vmax(b1, x);
        }
      }
      score[h] = g >= a.groups ? none : a.group_top == 2 && b2 > none ? b1 + b2 : b1;
      if (g < a.groups) lds_g[g] = score[h];
      if (F && b1 > none) size = vmax(size, vmax(b1, -b1) + (b2 > none ? vmax(b2, -b2) : V(0)));
    }
    wave_order();
    uint32_t kept = 0;
    V low = -none, high = none;  // the worst kept score, the best other one
    int better[H];
#pragma unroll
    for (int h = 0; h < H; ++h) better[h] = 0;
    for (int o = 0; o < a.groups; o += 4) {
      V v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = lds_g[min(o + u, a.groups - 1)];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int h = 0; h < H; ++h)
          better[h] += (o + u < a.groups) & ((v[u] > score[h]) | ((v[u] == score[h]) & (o + u < lane + LPT * h)));
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int g = lane + LPT * h;
      const bool keep = g < a.groups && better[h] < a.top_groups;
      if (keep) low = low < score[h] ? low : score[h];
      else high = vmax(high, score[h]);
      const uint64_t bits = __ballot(keep) >> (threadIdx.x / LPT * LPT);
      kept |= LPT == 64 ? static_cast<uint32_t>(bits) : static_cast<uint32_t>(bits & 0xFFFF) << (16 * h);
    }
    if constexpr (F) {
      low = -row_max<LPT>(-low);
      high = row_max<LPT>(high);
      // a sum of two is off by both, and by its own rounding
      if (unsure(low, high, group_exact, far, near, 2.0f * err + 2.0f * kRound * row_max<LPT>(size))) found = AGAIN;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = kept >> (grp[i] & 31) & 1 ? key[i] : none;
  }
  V last = -none, kth = -none;
  *id = kNoExpert;
  const int picks = F ? a.K + 2 : a.K;  // float: two more, to compare the last choice with
  for (int j = 0; j < picks; ++j) {
    V b = none;
#pragma unroll
    for (int i = 0; i < N; ++i) b = vmax(b, key[i]);
    b = row_max<LPT>(b);
    if constexpr (F) {
      // the K chosen are among the K + 1 best if the one after those is sure to be below the K-th
      const bool tie = j > 0 && unsure(j <= a.K ? last : kth, b, exact, far, near, err + kRound * fabsf(last));
      if (tie) found = max(found, exact || j > a.K ? static_cast<int>(AGAIN) : static_cast<int>(REORDER));
      if (j > a.K) break;
      if (j == a.K - 1) kth = b;
    }
    last = b;
    int e = kNoExpert;
#pragma unroll
    for (int i = N - 1; i >= 0; --i) e = key[i] == b ? 4 * LPT * (i / 4) + i % 4 : e;
    e = row_min<LPT>(e == kNoExpert || !(b > none) ? kNoExpert : e + 4 * lane);
    const int at = e - 4 * lane;
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = at == 4 * LPT * (i / 4) + i % 4 ? none : key[i];
    if (lane == j) *id = e;
  }
  return found;
}

template <int LPT, int Q, typename T>
__global__ __launch_bounds__(64) void route_grouped_kernel(GroupedRouteArgs a, int32_t* __restrict__ topk_idx,
                                                           float* __restrict__ topk_gate) {
  constexpr int TOK = 64 / LPT;
  constexpr int W = 4 * LPT * Q + kMaxGroups;
  __shared__ float lds32[TOK][W], lds32g[TOK][kMaxGroups];
  const int lane = threadIdx.x % LPT, tok = threadIdx.x / LPT;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * TOK + tok;
  const bool live = t < a.T;
  const T* row = static_cast<const T*>(a.logits) + t * a.E;
  float l[4 * Q];
  load_logits<LPT, Q>(row, a.E, lane, live, l);
  int id;
  const int found = choose<LPT, Q>(a, l, lane, lds32[tok], lds32g[tok], &id);
  uint64_t again = __ballot(found == AGAIN);
  if (__builtin_expect(again != 0, 0)) {  // token by token, by all 64 lanes
    constexpr int Q64 = (4 * LPT * Q + 255) / 256;
    __shared__ double lds64[256 * Q64 + kMaxGroups], lds64g[kMaxGroups];
    while (again != 0) {
      const int k = (__ffsll(static_cast<unsigned long long>(again)) - 1) / LPT;
      again &= LPT == 64 ? 0 : ~(uint64_t{0xFFFF} << (16 * k));
      float l64[4 * Q64];
      load_logits<64, Q64>(static_cast<const T*>(a.logits) + (static_cast<int64_t>(blockIdx.x) * TOK + k) * a.E, a.E,
                           threadIdx.x, true, l64);
      int id64;
      choose<64, Q64>(a, l64, threadIdx.x, lds64, lds64g, &id64);
      id64 = __shfl(id64, lane);
      if (tok == k) id = id64;
      wave_order();
    }
  }
  if (__builtin_expect(__ballot(found == REORDER) != 0, 0)) {  // scores with a bias
    const bool in = id != kNoExpert;
    double m = 0.0, sum = 1.0;
    if (!a.sigmoid) row_softmax<LPT, double, 4 * Q>(l, &m, &sum);
    const double x = in ? static_cast<double>(Elem<T>::load(row + id)) : 0.0;
    const double s = a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - m) * (1.0 / sum);
    const double c = in ? s + static_cast<double>(a.bias[id]) : -__builtin_huge_val();
    int rank = 0;
    for (int k = 0; k <= a.K; ++k) {
      const int from = (LPT == 64 ? 0 : static_cast<int>(threadIdx.x) & 48) + k;
      const double ck = __shfl(c, from);
      const int ik = __shfl(id, from);
      rank += ck > c || (ck == c && ik < id) ? 1 : 0;
    }
    // (choices that no expert is left for rank last, in any order: their ids are the same)
    int* const place = reinterpret_cast<int*>(lds32[tok]);
    if (lane <= a.K) place[lane] = kNoExpert;
    wave_order();
    if (in && lane <= a.K) place[rank] = id;
    wave_order();
    if (found == REORDER) id = lane <= a.K ? place[lane] : kNoExpert;
  }
  if (lane >= a.K) id = kNoExpert;
  // gates in float64 (one exponential per chosen expert)
  const bool got = id != kNoExpert;
  const double x = got && live ? static_cast<double>(Elem<T>::load(row + id)) : 0.0;
  double s = 0.0, D = 1.0;
  if (a.sigmoid) {
    s = got ? 1.0 / (1.0 + exp(-x)) : 0.0;
    if (a.renorm) D = fmax(row_sum<16>(s), 0x1p-126);
  } else {
    float m, sum;
    if (a.renorm) {
      m = row_max<16>(got ? static_cast<float>(x) : kNone);
      s = got ? exp(x - static_cast<double>(m)) : 0.0;
      D = row_sum<16>(s);
    } else {
      row_softmax<LPT, float, 4 * Q>(l, &m, &sum);
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
// Bound: the writes (T E values) for large batches. Measured: 16384 tokens of 256 experts, float32, 7.7 us = 2.4 TB/s with
// what a launch costs (3 us); 255 tokens of 64 experts, raw softmax gates, below the 8 us that a call takes on the host.
constexpr int kLanes = 16;         // lanes per token of the gradient
constexpr int kTok = 64 / kLanes;  // tokens per wave

template <int Q, typename T>
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
      const double D = fmax(row_sum<kLanes>(s), 0x1p-126), us = row_sum<kLanes>(got ? u * s : 0.0);
      ds = (u - us / D) / D;
    }
    v = ds * s * (1.0 / (1.0 + exp(x)));  // 1 - s without its cancellation
  } else if (a.renorm) {
    const double top = static_cast<double>(row_max<kLanes>(got ? static_cast<float>(x) : kNone));
    const double ex = got ? exp(x - top) : 0.0;
    const double D = row_sum<kLanes>(ex);
    const double gj = D > 0.0 ? ex / D : 0.0;
    v = gj * (u - row_sum<kLanes>(got ? gj * u : 0.0));
  } else {
    load_logits<kLanes, Q>(row, a.E, lane, live, l);
    row_softmax<kLanes, float, 4 * Q>(l, &m, &sum);
    if (sum != sum || sum == 0.0f) got = false, sum = 1.0f, m = -kNone;  // every score is 0 (or NaN): no gradient
    sum = 1.0f / sum;
    const double p = got ? exp(x - static_cast<double>(m)) * static_cast<double>(sum) : 0.0;
    v = got ? p * u : 0.0;
    dot = static_cast<float>(row_sum<kLanes>(v));
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

// f(Q) for Q = ceil(E / per) runs per lane, up to 8; 5 and 7 run as 6 and 8
template <typename F>
hipError_t by_width(int E, int per, F&& f) {
  switch ((E + per - 1) / per) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 3: return f(std::integral_constant<int, 3>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 5:
    case 6: return f(std::integral_constant<int, 6>{});
    default: return f(std::integral_constant<int, 8>{});
  }
}

// Up to this many tokens a wave takes one token where it has more than 64
// experts (up to 64, 16 lanes hold them four each as well). Measured, 64 lanes
// per token against 16: 256 experts in groups at 16 / 2048 / 4096 / 8192 tokens
// 7.0 / 9.2 / 12.4 / 19.5 us against 10.3 / 11.2 / 11.3 / 13.1; 512 experts at
// 2048 / 16384 tokens 10.5 / 45.8 against 16.2 / 36.8.
constexpr int kWaveTokens = 2048;

template <typename T>
hipError_t route(const GroupedRouteArgs& a, int32_t* topk_idx, float* topk_gate, hipStream_t st) {
  if (a.E > 64 && a.T <= kWaveTokens) {
    const dim3 grid(a.T), block(64);
    if (a.E <= 256) hipLaunchKernelGGL((route_grouped_kernel<64, 1, T>), grid, block, 0, st, a, topk_idx, topk_gate);
    else hipLaunchKernelGGL((route_grouped_kernel<64, 2, T>), grid, block, 0, st, a, topk_idx, topk_gate);
    return hipGetLastError();
  }
  return by_width(a.E, 64, [&](auto q) {
    hipLaunchKernelGGL((route_grouped_kernel<16, decltype(q)::value, T>), dim3((a.T + 3) / 4), dim3(64), 0, st, a,
                       topk_idx, topk_gate);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t route_backward(const GroupedRouteArgs& a, const int32_t* topk_idx, const float* dgate, void* dlogits,
                          hipStream_t st) {
  return by_width(a.E, 4 * kLanes, [&](auto q) {
    hipLaunchKernelGGL((route_grouped_bwd_kernel<decltype(q)::value, T>), dim3((a.T + kTok - 1) / kTok), dim3(64), 0, st,
                       a, topk_idx, dgate, static_cast<T*>(dlogits));
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_route_grouped(const GroupedRouteArgs& a, int32_t* topk_idx, float* topk_gate, hipStream_t st) {
  return a.bf16 ? route<bf16_t>(a, topk_idx, topk_gate, st) : route<float>(a, topk_idx, topk_gate, st);
}

hipError_t launch_route_grouped_backward(const GroupedRouteArgs& a, const int32_t* topk_idx, const float* dgate,
                                         void* dlogits, hipStream_t st) {
  return a.bf16 ? route_backward<bf16_t>(a, topk_idx, dgate, dlogits, st)
                : route_backward<float>(a, topk_idx, dgate, dlogits, st);
}

}  // namespace moe
