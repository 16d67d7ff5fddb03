// Grouped products of 8-bit operands with one power-of-two scale per block of
// 128, float32 sums, on the scaled matrix instructions of gfx950.
//
//   out[s][n] = sum over blocks b of 128 k of
//                 2^(xs[row(s)][b] - 127) 2^(ws_e[n / 128][b] - 127) sum_{k in b} x[row(s)][k] W_e[n][k]   (+ bias)
//
// e: the expert whose grouped rows hold s. Every value of an e4m3 x e4m3
// product is exact in float32; the instruction applies both scales (E8M0
// bytes), so a block costs no vector instruction for them.
#include "common.h"
#include "fp8.h"
#include "moe.h"

namespace moe {

namespace {

enum { F_F32 = 0, F_BF16 = 1, F_SWIGLU = 2, F_GELU = 3 };

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

struct Fp8Params {
  Fp8Gemm g;
  void* out;     // float32 or bfloat16 [S][N]; activation modes: e4m3 [S][N]
  uint8_t* qs;   // activation modes: scales [S][ceil(N / 128)]
  int n_mt;      // m-tiles of any grouping at most
};

// Scale byte of a block whose largest magnitude has the bits amax (448 = 1.75 2^8), and 2^(127 - byte).
__device__ __forceinline__ int scale_byte(uint32_t amax) {
  const int b = static_cast<int>(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(b, 0);
}
__device__ __forceinline__ float inverse_scale(int byte) { return __uint_as_float(static_cast<uint32_t>(254 - byte) << 23); }

// Owner of m-tile mt when every expert's rows are cut into tiles
// of bm rows, for up to 512 experts: lane l holds the tile counts of experts
// l P .. l P + P - 1 (P = ceil(E / 64)), a prefix sum over the lanes and a
// ballot find the lane, and the walk over its experts is wave-uniform. False
// when the grouping has no such tile.
__device__ __forceinline__ void rows_of(const Fp8Gemm& g, int e, int* beg, int* end) {
  if (g.offsets == nullptr) {
    *beg = 0;
    *end = g.S;
  } else {
    expert_rows(g.offsets, e, g.S, INT32_MAX, beg, end);
  }
}

__device__ __forceinline__ bool tile_owner(const Fp8Gemm& g, int bm, int mt, int* expert, int* row0, int* rows) {
  const int lane = threadIdx.x % 64;
  const int P = (g.E + 63) / 64;
  int n = 0;
  for (int i = 0; i < P; ++i) {
    const int e = lane * P + i;
    if (e < g.E) {
      int b, en;
      rows_of(g, e, &b, &en);
      n += (en - b + bm - 1) / bm;
    }
  }
  int incl = n;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(incl, o);
    if (lane >= o) incl += v;
  }
  const int l = __popcll(__ballot(incl <= mt));
  if (l >= 64) return false;
  int local = mt - (__shfl(incl, l) - __shfl(n, l));
  for (int i = 0; i < P; ++i) {
    const int e = __builtin_amdgcn_readfirstlane(l * P + i);
    if (e >= g.E) return false;
    int b, en;
    rows_of(g, e, &b, &en);
    const int t = (en - b + bm - 1) / bm;
    if (local < t) {
      *expert = e;
      *row0 = b + local * bm;
      *rows = min(bm, en - *row0);
      return true;
    }
    local -= t;
  }
  return false;
}

__device__ __forceinline__ float load_bias(const Fp8Gemm& g, int e, int n) {
  const size_t i = static_cast<size_t>(e) * g.N + n;
  return g.bias_bf16 ? bf16_to_f32(static_cast<const bf16_t*>(g.bias)[i]) : static_cast<const float*>(g.bias)[i];
}

// 32 bytes of a row at k (16-byte chunks past the end of the row read as zeros)
__device__ __forceinline__ i32x8_t load32(const uint8_t* row, int k, int Kd) {
  u32x4_t a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
  if (k < Kd) a = *reinterpret_cast<const u32x4_t*>(row + k);
  if (k + 16 < Kd) b = *reinterpret_cast<const u32x4_t*>(row + k + 16);
  return i32x8_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// Simple form: a block of four waves computes 32 grouped rows x 128 weight
// rows (one block of scales), each wave 32 of them, from global memory.
// v_mfma_scale_f32_32x32x64_f8f6f4 with the weights as the M operand: lane l
// gives 32 bytes of weight row l % 32 and of grouped row l % 32, and gets the
// products of grouped row l % 32 with weight rows 8 (r / 4) + 4 (l / 32) + r % 4.
template <int MODE>
__global__ __launch_bounds__(256) void gemm_fp8_kernel(Fp8Params p) {
  const Fp8Gemm& g = p.g;
  constexpr bool ACT = MODE == F_SWIGLU || MODE == F_GELU;
  constexpr int NMAT = MODE == F_SWIGLU ? 2 : 1;
  __shared__ uint32_t amax[4][32];
  int e, row0, rows;
  if (!tile_owner(g, 32, static_cast<int>(blockIdx.y), &e, &row0, &rows)) return;
  const int lane = threadIdx.x % 64, w = threadIdx.x / 64;
  const int kb = (g.Kd + kFp8Block - 1) / kFp8Block;
  const int nb = (g.N + kFp8Block - 1) / kFp8Block;
  const int n0 = static_cast<int>(blockIdx.x) * kFp8Block + w * 32;
  const int s = row0 + min(lane % 32, rows - 1);
  const int xr = g.rows != nullptr ? min(max(g.rows[s], 0), g.x_rows - 1) : s;
  const uint8_t* xrow = g.x + static_cast<size_t>(xr) * g.Kd;
  const uint8_t* xsrow = g.xs + static_cast<size_t>(xr) * kb;
  const int n = min(n0 + lane % 32, g.N - 1);
  const size_t wr = (static_cast<size_t>(e) * g.N + n) * g.Kd;
  const size_t wsr = (static_cast<size_t>(e) * nb + blockIdx.x) * kb;
  const uint8_t* wrow[2] = {g.W + wr, NMAT == 2 ? g.W3 + wr : nullptr};
  const uint8_t* wsrow[2] = {g.Ws + wsr, NMAT == 2 ? g.W3s + wsr : nullptr};
  f32x16_t acc[NMAT];
#pragma unroll
  for (int m = 0; m < NMAT; ++m)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[m][r] = 0.0f;
  for (int b = 0; b < kb; ++b) {
    const int sx = xsrow[b];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int k = b * kFp8Block + u * 64 + lane / 32 * 32;
      const i32x8_t x = load32(xrow, k, g.Kd);
#pragma unroll
      for (int m = 0; m < NMAT; ++m)
        acc[m] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(load32(wrow[m], k, g.Kd), x, acc[m], 0, 0, 0,
                                                                 static_cast<int>(wsrow[m][b]), 0, sx);
    }
  }
  const int ro = row0 + lane % 32;
  const bool live = lane % 32 < rows;
  float v[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int c = n0 + 8 * (r / 4) + 4 * (lane / 32) + r % 4;
    v[r] = acc[0][r];
    if (g.bias != nullptr && c < g.N) v[r] += load_bias(g, e, c);
    if (MODE == F_SWIGLU) v[r] = silu(v[r]) * acc[NMAT - 1][r];
    if (MODE == F_GELU) v[r] = gelu_exact(v[r]);
    if (ACT && c >= g.N) v[r] = 0.0f;
  }
  if constexpr (ACT) {
    float m = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) m = fmaxf(m, fabsf(v[r]));
    m = fmaxf(m, __shfl_xor(m, 32));
    if (lane < 32) amax[w][lane] = __float_as_uint(m);
    __syncthreads();
    uint32_t mm = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) mm = max(mm, amax[i][lane % 32]);
    const int b = scale_byte(mm);
    const float f = inverse_scale(b);
    if (!live) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = n0 + 8 * q + 4 * (lane / 32);
      if (c >= g.N) continue;
      int pk = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * q] * f, v[4 * q + 1] * f, 0, false);
      pk = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * q + 2] * f, v[4 * q + 3] * f, pk, true);
      *reinterpret_cast<int*>(static_cast<uint8_t*>(p.out) + static_cast<size_t>(ro) * g.N + c) = pk;
    }
    if (w == 0 && lane < 32) p.qs[static_cast<size_t>(ro) * nb + blockIdx.x] = static_cast<uint8_t>(b);
  } else {
    if (!live) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = n0 + 8 * q + 4 * (lane / 32);
      if (c >= g.N) continue;
      const size_t o = static_cast<size_t>(ro) * g.N + c;
      if (MODE == F_F32)
        *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.out) + o) =
            f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      else
        *reinterpret_cast<u32x2_t*>(static_cast<bf16_t*>(p.out) + o) =
            u32x2_t{pack_bf16x2(v[4 * q], v[4 * q + 1]), pack_bf16x2(v[4 * q + 2], v[4 * q + 3])};
    }
  }
}

template <int MODE>
hipError_t launch(const Fp8Gemm& g, void* out, uint8_t* qs, hipStream_t st) {
  Fp8Params p{g, out, qs, 0};
  p.n_mt = g.S / 32 + min(g.E, g.S);
  const dim3 grid((g.N + kFp8Block - 1) / kFp8Block, static_cast<unsigned>(p.n_mt));
  hipLaunchKernelGGL(gemm_fp8_kernel<MODE>, grid, dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_fp8(const Fp8Gemm& g, int out_type, void* out, hipStream_t st) {
  return out_type == FP8_OUT_F32 ? launch<F_F32>(g, out, nullptr, st) : launch<F_BF16>(g, out, nullptr, st);
}

size_t fp8_act_tmp_bytes(int64_t S, int64_t N, int64_t max_rows) { return 0; }

hipError_t launch_gemm_fp8_act(const Fp8Gemm& g, int act, uint8_t* q, uint8_t* qs, void* tmp, hipStream_t st) {
  return act == MOE_ACT_SWIGLU ? launch<F_SWIGLU>(g, q, qs, st) : launch<F_GELU>(g, q, qs, st);
}

}  // namespace moe
