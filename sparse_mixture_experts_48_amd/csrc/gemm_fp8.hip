// Grouped products of 8-bit operands with one power-of-two scale per block of
// 128, float32 sums, on the scaled matrix instructions of gfx950.
//
//   out[s][n] = sum over blocks b of 128 k of
//                 2^(xs[row(s)][b] - 127) 2^(ws_e[n / 128][b] - 127) sum_{k in b} x[row(s)][k] W_e[n][k]   (+ bias)
//
// e: the expert whose grouped rows hold s. Every value of an e4m3 x e4m3
// product is exact in float32; the instruction applies both scales (E8M0
// bytes), so a block costs no vector instruction for them.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "fp8.h"
#include "moe.h"
#include "quant_fp8.h"

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
  float* parts;  // split tiles: float32 sums of their parts, [part][split tile][BM][kBN]
};

// Buffer resource over `bytes` bytes at `base` (raw dword buffer; loads at
// byte offsets >= bytes return zeros).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0),
                                           static_cast<int>(bytes), 0x00020000);
}

// B bytes (4 or 16) per lane at byte offset voff + soff of the buffer into
// LDS: the wave writes 64 x B consecutive bytes at lds_wave_base. AUX 2: non-temporal.
template <int B, int AUX = 0>
__device__ __forceinline__ void lds_load(__amdgpu_buffer_rsrc_t r, uint32_t voff, int soff, void* lds_wave_base) {
  typedef __attribute__((address_space(3))) void lds_void;
  if constexpr (B == 16)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds_wave_base, 16, static_cast<int>(voff), soff, 0, AUX);
  else
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds_wave_base, 4, static_cast<int>(voff), soff, 0, AUX);
}

// s_waitcnt immediates (gfx9 encoding): vmcnt <= n only; that and lgkmcnt 0; lgkmcnt 0 only.
constexpr int vmcnt_imm(int n) { return (n & 0xF) | ((n >> 4) << 14) | (0x7 << 4) | (0xF << 8); }
constexpr int vmcnt_lgkm0_imm(int n) { return (n & 0xF) | ((n >> 4) << 14) | (0x7 << 4); }
constexpr int kLgkm0 = 0xF | (3 << 14) | (0x7 << 4);

// GELU(x) = x Phi(x), with Phi(-|x|) = e^(-x^2 / 2) R(|x|), R(x) = erfc(x / sqrt 2) e^(x^2 / 2) / 2 as a polynomial in
// t = 1 / (1 + 0.3 x): a minimax fit over 0 .. 14 by reweighted least squares, within 8.3e-6 of R, and 1.4e-5 of GELU in
// float32 arithmetic, tails included (the value is rounded to e4m3, by up to 2^-4, next). About 20 instructions without a
// branch; with erff instead, and the bias read one value at a time, the GELU layer of 4096 tokens (d 4096, width 14336)
// took 1181 us, with this 1056.
__device__ __forceinline__ float gelu(float x) {
  const float a = fabsf(x);
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3f, a, 1.0f));
  float p = -0.07709822803735733f;
  p = fmaf(p, t, 0.2160392552614212f);
  p = fmaf(p, t, -0.016950350254774094f);
  p = fmaf(p, t, 0.1441975086927414f);
  p = fmaf(p, t, 0.1137416660785675f);
  p = fmaf(p, t, 0.12007425725460052f);
  const float q = p * t * __builtin_amdgcn_exp2f(a * a * -0.72134752f);
  return x * (x >= 0.0f ? 1.0f - q : q);
}

// Store through a pointer the compiler knows to be global: stores through a
// generic pointer may write LDS, and then every later LDS read waits for them.
template <typename T>
__device__ __forceinline__ void store_global(void* ptr, T v) {
  *(__attribute__((address_space(1))) T*)(ptr) = v;
}

__device__ __forceinline__ void rows_of(const Fp8Gemm& g, int e, int* beg, int* end) {
  if (g.offsets == nullptr) {
    *beg = 0;
    *end = g.S;
  } else {
    expert_rows(g.offsets, e, g.S, INT32_MAX, beg, end);
  }
}

// Every expert's rows cut into m-tiles of bm rows, for up to 512 experts: lane
// l counts the tiles of experts l P .. l P + P - 1 (P = ceil(E / 64)), and a
// prefix sum over the lanes numbers them. All lanes of the wave take part.
struct MTiles {
  int n, incl;   // tiles of this lane's experts; and of those up to and including them
  int beg, end;  // rows of this lane's (last) expert
  int total;     // all tiles (wave-uniform)
};
__device__ __forceinline__ MTiles count_tiles(const Fp8Gemm& g, int bm) {
  const int lane = threadIdx.x % 64;
  const int P = (g.E + 63) / 64;
  MTiles t{0, 0, 0, 0, 0};
  for (int i = 0; i < P; ++i) {
    const int e = lane * P + i;
    rows_of(g, min(e, g.E - 1), &t.beg, &t.end);
    t.n += e < g.E ? (t.end - t.beg + bm - 1) / bm : 0;
  }
  t.incl = t.n;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(t.incl, o);
    if (lane >= o) t.incl += v;
  }
  t.total = __builtin_amdgcn_readfirstlane(__shfl(t.incl, 63));
  return t;
}

// Owner of m-tile mt (0 <= mt < total): a ballot finds its lane; with more
// than 64 experts the walk over that lane's experts is wave-uniform.
__device__ __forceinline__ void tile_owner(const Fp8Gemm& g, const MTiles& t, int bm, int mt, int* expert, int* row0,
                                           int* rows) {
  const int P = (g.E + 63) / 64;
  const int l = __popcll(__ballot(t.incl <= mt));
  int local = __builtin_amdgcn_readfirstlane(mt - (__shfl(t.incl, l) - __shfl(t.n, l)));
  int e = l, b = __shfl(t.beg, l), en = __shfl(t.end, l);
  if (P > 1) {
    for (int i = 0; i < P; ++i) {
      e = __builtin_amdgcn_readfirstlane(min(l * P + i, g.E - 1));
      rows_of(g, e, &b, &en);
      const int n = (en - b + bm - 1) / bm;
      if (local < n) break;
      local -= n;
    }
  }
  *expert = __builtin_amdgcn_readfirstlane(e);
  *row0 = __builtin_amdgcn_readfirstlane(b + local * bm);
  *rows = __builtin_amdgcn_readfirstlane(min(bm, en - (b + local * bm)));
}

// Most m-tiles that S rows of E experts can have.
int64_t most_tiles(const Fp8Gemm& g, int bm) { return g.S <= g.E ? g.S : g.E + (g.S - g.E) / bm; }

// bias of columns n .. n + 3 (n and N are multiples of 4)
__device__ __forceinline__ f32x4_t load_bias(const Fp8Gemm& g, int e, int n) {
  const size_t i = static_cast<size_t>(e) * g.N + n;
  if (!g.bias_bf16) return *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(g.bias) + i);
  const u32x2_t v = *reinterpret_cast<const u32x2_t*>(static_cast<const bf16_t*>(g.bias) + i);
  return f32x4_t{__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xFFFF0000u), __uint_as_float(v[1] << 16),
                 __uint_as_float(v[1] & 0xFFFF0000u)};
}

// ---------------------------------------------------------------------------- tiled kernel
//
// A block of 8 waves (WM x WN) computes BM grouped rows x BN = 256 weight rows
// (SwiGLU: 128 rows of W1 and the same 128 of W3) on
// v_mfma_scale_f32_32x32x64_f8f6f4, the weights as the M operand: lane l gives
// 32 bytes of weight row l % 32 and of grouped row l % 32 (k 32 (l / 32) .. of
// the step's 64; both operands agree on which k a byte holds), and gets the
// products of grouped row l % 32 with weight rows 8 (r / 4) + 4 (l / 32) + r % 4.
//
// k is staged 128 at a time, one block of scales and one 128-byte line of
// every row: direct global-to-LDS loads fill a ring of NAS slots (256 rows: two,
// 128 rows: three), NAS - 1 stages ahead. LDS rows are eight 16-byte chunks,
// chunk c of row r at c ^ key(r), so that the fragment reads of 8 or 16
// consecutive rows fall in distinct bank groups. Rows past the last
// repeat it (their products are not stored); past the end of k (a multiple of
// 16) loads take an offset past the buffer and read zeros.
//
// Scales: the bytes of up to kSC blocks of every row of the tile sit in LDS as
// dwords of four consecutive blocks, [group of 4][row]; a stage reads one dword
// per 32 rows and shifts its byte down. The instruction applies both bytes.
//
// Measured: 8192 rows of 8 experts, N 2 x 14336, Kd 4096 (SwiGLU) 849 us = 2.27 PFLOP/s, N 4096, Kd 14336 461 us = 2.09;
// dense 8192 rows, N 4096, Kd 4096 108 us = 2.54. No single bound: of a CU's busy cycles (at 1.97 GHz) the MFMAs take 51 %
// and the fragment reads from LDS 28 % (6 % of those for conflicts, all outside the main loop); timed without the global
// loads a stage took 0.73 of its time, with all of them from one tile 0.92, without the fragment reads 0.9. A second
// block per CU would run through the first one's stalls, but LDS holds one.
constexpr int kBK = 128;   // k per stage: one block of scales
constexpr int kCH = 8;     // 16-byte chunks per LDS row
// blocks of scales held in LDS at once: a multiple of 4 and of the ring's length
template <int BM> constexpr int kScaleBlocks = BM == 256 ? 112 : 108;
constexpr int kBN = 256;   // weight rows per tile
constexpr int kTileGroupN = 4;  // n-tiles per group in the XCD-aware order

__device__ __forceinline__ int swz_key(int row) { return (row & 7) ^ ((row >> 3) & 1); }
__device__ __forceinline__ int swz(int row, int chunk) { return row * kCH + (chunk ^ swz_key(row)); }

__device__ __forceinline__ i32x8_t join(u32x4_t a, u32x4_t b) {
  return __builtin_bit_cast(i32x8_t, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// SPLIT (float32 output): the tiles past the last full round of one per CU are
// each cut along the reduction into parts that fill about one more round of
// short blocks (tile_split); their float32 sums go to scratch and sum_parts_kernel
// adds them in order.
struct TileSplit {
  int full;   // tiles that run whole
  int rest;   // tiles after them, in `parts` parts each
  int parts;
};
constexpr int kCUs = 256;
constexpr int kMaxParts = 8, kPartStages = 8;  // parts of a tile at most, stages of a part at least
__device__ __forceinline__ TileSplit tile_split(int n_t, int KB) {
  const int rest = n_t % kCUs;
  const int parts = rest > 0 ? min(min(kCUs / rest, kMaxParts), KB / kPartStages) : 1;
  return parts > 1 ? TileSplit{n_t - rest, rest, parts} : TileSplit{n_t, 0, 1};
}

// Tile t of n_nt x n_mt, ordered (group of n-tiles) x (m-tile) x (n-tile in group).
__device__ __forceinline__ void tile_place(int t, int n_nt, int n_mt, int* mt, int* nt) {
  const int gr = t / (kTileGroupN * n_mt);
  const int gs = min(kTileGroupN, n_nt - gr * kTileGroupN);
  const int rem = t - gr * kTileGroupN * n_mt;
  *mt = rem / gs;
  *nt = gr * kTileGroupN + rem % gs;
}

template <int BM, int MODE, bool SPLIT>
__global__ __launch_bounds__(512) void gemm_fp8_tile_kernel(Fp8Params p) {
  static_assert(!SPLIT || MODE == F_F32, "parts are float32 sums");
  constexpr bool ACT = MODE == F_SWIGLU || MODE == F_GELU;
  constexpr int NMAT = MODE == F_SWIGLU ? 2 : 1;
  constexpr int WM = BM / 64, WN = 8 / WM;     // waves: each 64 grouped rows x BN / WN weight rows
  constexpr int WTN = kBN / WN;
  constexpr int TM = 2, TN = WTN / 32;         // 32 x 32 accumulators of a wave
  constexpr int TNO = TN / NMAT;               // column tiles of its output
  constexpr int NAS = BM == 256 ? 2 : 3;       // ring slots
  constexpr int A_IN = BM / 64, B_IN = kBN / 64;  // loads per wave and stage (8 rows each)
  // loads per sub-step: on 256 rows all of them in the first half of a stage (they are due at its end); measured on the
  // prefill layer 1, 2, 4, 8 per sub-step: 1538, 1470, 1484, 1511 us
  constexpr int PER = BM == 256 ? 2 : (A_IN + B_IN + 2 * TN - 1) / (2 * TN);
  constexpr int WAITN = (NAS - 2) * (A_IN + B_IN);
  constexpr int NCOLS = kBN / NMAT;
  constexpr int kSC = kScaleBlocks<BM>;
  __shared__ u32x4_t A0[BM * kCH], A1[BM * kCH];
  __shared__ u32x4_t B0[kBN * kCH], B1[kBN * kCH];
  __shared__ uint32_t XS[kSC / 4 * BM];            // [group of 4 blocks][row]
  __shared__ uint32_t WS[2 * 32];              // [block of weight rows][group of 4 blocks]
  u32x4_t *A2 = A0, *B2 = B0;
  if constexpr (NAS == 3) {
    __shared__ u32x4_t A2s[BM * kCH], B2s[kBN * kCH];
    A2 = A2s;
    B2 = B2s;
  }
  u32x4_t* const as[3] = {A0, A1, A2};
  u32x4_t* const bs[3] = {B0, B1, B2};

  const Fp8Gemm& g = p.g;
  const int lane = threadIdx.x % 64;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int wm = wid / WN, wn = wid % WN;
  const int Kd = g.Kd, N = g.N;
  const int KB = (Kd + kBK - 1) / kBK, NB = (N + kBK - 1) / kBK;

  // Tile order: block b runs on XCD b % 8; every XCD takes a contiguous run of
  // tiles, so that blocks that run together share rows and weights in that XCD's
  // L2, and after them a run of the parts of split tiles (part by part).
  const int n_nt = (N + NCOLS - 1) / NCOLS;
  const MTiles mtiles = count_tiles(g, BM);
  const int n_mt = min(p.n_mt, mtiles.total);
  const int n_t = n_nt * n_mt;
  const TileSplit sp = SPLIT ? tile_split(n_t, KB) : TileSplit{n_t, 0, 1};
  const int xcd = static_cast<int>(blockIdx.x % 8), at = static_cast<int>(blockIdx.x / 8);
  const int per_xcd = (sp.full + 7) / 8;
  int t = xcd * per_xcd + at;
  int kt0 = 0, kt1 = KB;     // this block's stages
  int slot = -1, part = 0;   // its place in p.parts (-1: a whole tile)
  if (!SPLIT || at < per_xcd) {
    if (at >= per_xcd || t >= sp.full) return;
  } else {
    const int n_p = sp.rest * sp.parts, per = (n_p + 7) / 8;
    slot = xcd * per + at - per_xcd;
    if (at - per_xcd >= per || slot >= n_p) return;
    part = slot / sp.rest;
    t = sp.full + slot - part * sp.rest;
    const int q = ((KB + sp.parts - 1) / sp.parts + 3) / 4 * 4;  // (scales are loaded four blocks at a time)
    kt0 = min(KB, part * q);
    kt1 = min(KB, kt0 + q);
  }
  int mt, nt;
  tile_place(t, n_nt, n_mt, &mt, &nt);
  const int n0 = nt * NCOLS;
  int e = 0, row0 = 0, rows = 0;
  tile_owner(g, mtiles, BM, mt, &e, &row0, &rows);

  const uint32_t a_bytes = static_cast<uint32_t>(g.x_rows) * static_cast<uint32_t>(Kd);
  const uint32_t b_bytes = static_cast<uint32_t>(N) * static_cast<uint32_t>(Kd);
  const __amdgpu_buffer_rsrc_t ra = buffer_rsrc(g.x, a_bytes);
  __amdgpu_buffer_rsrc_t rb1 = ra, rb3 = ra;
  const int k_last = (KB - 1) * kBK;  // first k of the last stage
  auto x_row = [&](int r) {           // row of x of the tile's row r
    const int s = row0 + min(r, rows - 1);
    return g.rows != nullptr ? min(max(g.rows[s], 0), g.x_rows - 1) : s;
  };
  // byte offsets of the lane's loads: for every stage, and for the last one
  uint32_t a_vo[A_IN], a_vl[A_IN], b_vo[B_IN], b_vl[B_IN];
  auto setup = [&]() {
    rb1 = buffer_rsrc(g.W + static_cast<size_t>(e) * N * Kd, b_bytes);
    if constexpr (NMAT == 2) rb3 = buffer_rsrc(g.W3 + static_cast<size_t>(e) * N * Kd, b_bytes);
#pragma unroll
    for (int u = 0; u < A_IN; ++u) {
      const int r = (wid * A_IN + u) * 8 + lane / 8;
      const int kc = ((lane % 8) ^ swz_key(r)) * 16;
      a_vo[u] = static_cast<uint32_t>(x_row(r)) * static_cast<uint32_t>(Kd) + static_cast<uint32_t>(kc);
      a_vl[u] = k_last + kc < Kd ? a_vo[u] : a_bytes;
    }
#pragma unroll
    for (int u = 0; u < B_IN; ++u) {
      const int r = (wid * B_IN + u) * 8 + lane / 8;
      const int kc = ((lane % 8) ^ swz_key(r)) * 16;
      // SwiGLU: rows are, per wave column, WTN / 2 of W1, then the same of W3
      const int c = NMAT == 2 ? r / WTN * (WTN / 2) + r % (WTN / 2) : r;
      const int n = min(n0 + c, N - 1);
      b_vo[u] = static_cast<uint32_t>(n) * static_cast<uint32_t>(Kd) + static_cast<uint32_t>(kc);
      b_vl[u] = k_last + kc < Kd ? b_vo[u] : b_bytes;
    }
  };
  auto load_a = [&](int u, int k0, u32x4_t* As) {
    lds_load<16>(ra, k0 >= k_last ? a_vl[u] : a_vo[u], min(k0, k_last), As + (wid * A_IN + u) * 64);
  };
  auto load_b = [&](int u, int k0, u32x4_t* Bs) {
    const bool third = NMAT == 2 && (wid * B_IN + u) * 8 % WTN >= WTN / 2;  // the 8 rows share a matrix
    lds_load<16>(third ? rb3 : rb1, k0 >= k_last ? b_vl[u] : b_vo[u], min(k0, k_last), Bs + (wid * B_IN + u) * 64);
  };
  // Scales of blocks c0 .. c0 + kSC - 1 of the tile's rows into LDS. Direct
  // loads of whole dwords where rows of scales start on one, else bytes.
  auto load_scales = [&](int c0) {
    const int nblk = min(kSC, kt1 - c0), ng = (nblk + 3) / 4;
    const uint32_t xb = static_cast<uint32_t>(g.x_rows) * static_cast<uint32_t>(KB);
    // weights: one row of blocks per (matrix or half of the tile); lane 32 h + i takes dword i of half h
    const int h = lane / 32, i4 = lane % 32 * 4;
    const uint8_t* wsr = (NMAT == 2 && h ? g.W3s : g.Ws) +
                         (static_cast<size_t>(e) * NB + min(n0 / kBK + (NMAT == 1 ? h : 0), NB - 1)) * KB + c0;
    if (wid == 0) {
      uint32_t v = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (i4 + q < nblk) v |= static_cast<uint32_t>(wsr[i4 + q]) << (8 * q);
      WS[lane] = v;
    }
    if (KB % 4 == 0 && c0 % 4 == 0) {
      const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(g.xs, xb);
      for (int q = wid; q < ng * (BM / 64); q += 8) {
        const int gq = q / (BM / 64), rq = q % (BM / 64) * 64;
        lds_load<4>(rs, static_cast<uint32_t>(x_row(rq + lane)) * static_cast<uint32_t>(KB), c0 + gq * 4, XS + gq * BM + rq);
      }
    } else {
      for (int q = wid; q < ng * (BM / 64); q += 8) {
        const int gq = q / (BM / 64), r = q % (BM / 64) * 64 + lane;
        const uint8_t* xr = g.xs + static_cast<size_t>(x_row(r)) * KB + c0;
        uint32_t v = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (gq * 4 + b < nblk) v |= static_cast<uint32_t>(xr[gq * 4 + b]) << (8 * b);
        XS[gq * BM + r] = v;
      }
    }
  };

  f32x16_t acc[TN][TM];
  const int frow = lane % 32, fsub = lane / 32;
  auto run_stage = [&](auto mf, int kt, int sblk, const u32x4_t* As, const u32x4_t* Bs, u32x4_t* Bn, u32x4_t* An) {
    constexpr bool MF = decltype(mf)::value;
    // this wave's loads of the stage have landed, and its LDS reads of the last
    // stage are done (after the barrier other waves refill those slots, and the
    // barrier itself waits for no read in flight)
    __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(WAITN));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();  // ... and every wave's
    asm volatile("" ::: "memory");
    // Sub-step u = (64-k step u / TN, column tile u % TN): two MFMAs. Weight
    // fragments are read two sub-steps ahead (three buffers of 8 registers),
    // row fragments one step ahead; all of a step's fragments two deep would
    // not fit beside the 128 accumulators.
    constexpr int NU = 2 * TN;
    i32x8_t wf[3], xf[2][TM];
    int sx[TM], sw[NMAT];
    auto read_w = [&](int u) {
      const int r = wn * WTN + u % TN * 32 + frow, c = u / TN * 4 + fsub * 2;
      wf[u % 3] = join(Bs[swz(r, c)], Bs[swz(r, c + 1)]);
    };
    auto read_x = [&](int ks) {
      const int c = ks * 4 + fsub * 2;
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int r = wm * 64 + i * 32 + frow;
        xf[ks][i] = join(As[swz(r, c)], As[swz(r, c + 1)]);
      }
    };
    if constexpr (MF) {
      read_x(0);
      read_w(0);
#pragma unroll
      for (int i = 0; i < TM; ++i) sx[i] = static_cast<int>(XS[sblk / 4 * BM + wm * 64 + i * 32 + frow] >> (sblk % 4 * 8));
#pragma unroll
      for (int m = 0; m < NMAT; ++m)
        sw[m] = static_cast<int>(WS[(NMAT == 2 ? m : wn * WTN / 128) * 32 + sblk / 4] >> (sblk % 4 * 8));
      read_w(1);
    }
#pragma unroll
    for (int u = 0; u < NU; ++u) {
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        const int idx = u * PER + q;
        if (idx < B_IN) load_b(idx, (kt + NAS - 1) * kBK, Bn);
        else if (idx < A_IN + B_IN) load_a(idx - B_IN, (kt + NAS - 1) * kBK, An);
      }
      asm volatile("" ::: "memory");  // keep the loads ahead of the later fragment reads
      if constexpr (MF) {
        if (u == TN - 2) read_x(1);
        if (u + 2 < NU) read_w(u + 2);
        const int ks = u / TN, j = u % TN;
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < TM; ++i)
          acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[u % 3], xf[ks][i], acc[j][i], 0, 0, 0,
                                                                      sw[j / TNO], 0, sx[i]);
        __builtin_amdgcn_s_setprio(0);
      }
    }
  };
  // stages 0 .. NAS - 2 of the tile
  auto prologue = [&]() {
#pragma unroll
    for (int j = 0; j < NAS - 1; ++j) {
#pragma unroll
      for (int u = 0; u < B_IN; ++u) load_b(u, (kt0 + j) * kBK, bs[j]);
#pragma unroll
      for (int u = 0; u < A_IN; ++u) load_a(u, (kt0 + j) * kBK, as[j]);
    }
  };
  auto ring = [&](auto mf) {
    for (int c0 = kt0; c0 < kt1; c0 += kSC) {
      if (c0 > kt0) {  // the next blocks of scales: every wave has read the last ones
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        load_scales(c0);
        __builtin_amdgcn_s_waitcnt(kLgkm0);
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
        asm volatile("" ::: "memory");
      }
      const int c1 = min(kt1, c0 + kSC);
      int kt = c0;
      for (; kt + NAS <= c1; kt += NAS) {
#pragma unroll
        for (int i = 0; i < NAS; ++i)
          run_stage(mf, kt + i, kt + i - c0, as[i], bs[i], bs[(i + NAS - 1) % NAS], as[(i + NAS - 1) % NAS]);
      }
      // only the last group of blocks may end inside a period (kSC is a multiple of both ring lengths)
#pragma unroll
      for (int i = 0; i + 1 < NAS; ++i)
        if (kt + i < c1) run_stage(mf, kt + i, kt + i - c0, as[i], bs[i], bs[(i + NAS - 1) % NAS], as[(i + NAS - 1) % NAS]);
    }
  };

  // The wave's 32 rows of output tile i leave through LDS, in runs of 16 bytes: a lane holds four columns of one row, and
  // stores straight from there touch 32 rows each. Chunk c of row r is kept at c ^ (r % NCH). Measured, direct stores
  // against these: 16 experts of 512 rows, N 2048, Kd 1024 45 / 36 us; 64 of 128, N 4096, Kd 1376 147 / 140; the prefill
  // layer 1408 / 1375.
  constexpr int ES = ACT ? 1 : MODE == F_BF16 ? 2 : 4;
  constexpr int CW = WTN / NMAT;     // output columns of a wave
  constexpr int NCH = CW * ES / 16;  // 16-byte chunks of a row
  u32x4_t* const mine = BM == 256 ? (wid < 4 ? (wid < 2 ? A0 : A1) : (wid < 6 ? B0 : B1)) + wid % 2 * 1024
                                  : (wid < 4 ? B0 : B1) + wid % 4 * 512;
  static_assert(32 * NCH <= (BM == 256 ? 1024 : 512), "a wave's rows fit its place");
  auto order = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  };
  auto rows_out = [&](int i, int cw, char* dst) {  // dst: the wave's column cw of the tile's row 0; rows of N or kBN columns
    order();
    const size_t stride = static_cast<size_t>(SPLIT && slot >= 0 ? kBN : N) * ES;
#pragma unroll
    for (int t = 0; t < NCH / 2; ++t) {
      const int c = t * 64 + lane, row = c / NCH, ch = c % NCH;
      const u32x4_t v = mine[row * NCH + (ch ^ (row % NCH))];
      const int r = wm * 64 + i * 32 + row;
      if (r < rows && cw + ch * (16 / ES) < N) store_global(dst + r * stride + ch * 16, v);
    }
    order();
  };
  auto epilogue = [&]() {
    const int cw = n0 + wn * CW;  // the wave's first output column
    if (g.bias != nullptr && part == 0) {
#pragma unroll
      for (int j = 0; j < TNO; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4_t b = load_bias(g, e, min(cw + j * 32 + q * 8 + fsub * 4, N - 4));
#pragma unroll
          for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[j][i][4 * q + c] += b[c];
          if (q == 3) __builtin_amdgcn_sched_barrier(0);  // four loads in flight, not all of the tile's
        }
    }
    if constexpr (ACT) {
      // the activation, 0 past the last column; its largest magnitude per row
      float am[TM];
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        am[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < TNO; ++j)
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            float v = acc[j][i][q];
            v = MODE == F_SWIGLU ? silu(v) * acc[j + TN - TNO][i][q] : gelu(v);
            if (cw + j * 32 + q / 4 * 8 + fsub * 4 >= N) v = 0.0f;
            acc[j][i][q] = v;
            am[i] = fmaxf(am[i], fabsf(v));
            // a few activations at a time: interleaved over all 64, their temporaries spilled
            if (MODE == F_GELU ? q % 2 == 1 : q % 4 == 3) __builtin_amdgcn_sched_barrier(0);
          }
        am[i] = fmaxf(am[i], __shfl_xor(am[i], 32));
      }
      // the waves that share a row and a block of 128 columns (SwiGLU: every wave
      // column; GELU: those of the same half) exchange their maxima
      constexpr int SHARE = MODE == F_SWIGLU ? WN : WN / 2;
      uint32_t m[TM];
#pragma unroll
      for (int i = 0; i < TM; ++i) m[i] = __float_as_uint(am[i]);
      if constexpr (SHARE > 1) {
        __shared__ uint32_t red[WN * BM];
        if (fsub == 0) {
#pragma unroll
          for (int i = 0; i < TM; ++i) red[wn * BM + wm * 64 + i * 32 + frow] = m[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int v = 0; v < SHARE; ++v) m[i] = max(m[i], red[(wn / SHARE * SHARE + v) * BM + wm * 64 + i * 32 + frow]);
      }
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        if (wm * 64 + i * 32 >= rows) continue;
        const int r = wm * 64 + i * 32 + frow;
        const int b = scale_byte(m[i]);
        const float f = inverse_scale(b);
#pragma unroll
        for (int j = 0; j < TNO; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            int pk = __builtin_amdgcn_cvt_pk_fp8_f32(acc[j][i][4 * q] * f, acc[j][i][4 * q + 1] * f, 0, false);
            pk = __builtin_amdgcn_cvt_pk_fp8_f32(acc[j][i][4 * q + 2] * f, acc[j][i][4 * q + 3] * f, pk, true);
            reinterpret_cast<int*>(mine + frow * NCH + ((j * 2 + q / 2) ^ (frow % NCH)))[q % 2 * 2 + fsub] = pk;
          }
        rows_out(i, cw, static_cast<char*>(p.out) + static_cast<size_t>(row0) * N + cw);
        const int blk = cw / kBK;
        if (wn % SHARE == 0 && fsub == 0 && blk < NB && r < rows)
          store_global(p.qs + static_cast<size_t>(row0 + r) * NB + blk, static_cast<uint8_t>(b));
      }
    } else {
      char* const dst = SPLIT && slot >= 0
          ? reinterpret_cast<char*>(p.parts + static_cast<size_t>(slot) * BM * kBN + (cw - n0))
          : static_cast<char*>(p.out) + (static_cast<size_t>(row0) * N + cw) * ES;
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        if (wm * 64 + i * 32 >= rows) continue;
#pragma unroll
        for (int j = 0; j < TNO; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float v[4] = {acc[j][i][4 * q], acc[j][i][4 * q + 1], acc[j][i][4 * q + 2], acc[j][i][4 * q + 3]};
            if constexpr (MODE == F_F32)
              mine[frow * NCH + ((j * 8 + q * 2 + fsub) ^ (frow % NCH))] = __builtin_bit_cast(u32x4_t, f32x4_t{v[0], v[1], v[2], v[3]});
            else
              reinterpret_cast<u32x2_t*>(mine + frow * NCH + ((j * 4 + q) ^ (frow % NCH)))[fsub] =
                  u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
          }
        rows_out(i, cw, dst);
      }
    }
  };

  setup();
  load_scales(kt0);
  prologue();
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.0f;
  __builtin_amdgcn_s_waitcnt(kLgkm0);  // scales written by this wave
  if (wm * 64 < rows) ring(std::true_type{});
  else ring(std::false_type{});        // no rows of the tile: only its share of the loads
  // every wave's loads have landed and its LDS reads are done: the ring's slots carry the output now
  __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(0));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  epilogue();
}

// out = the sums of the split tiles' parts, in the order 0, 1, ...: blocks of 8 rows of a tile.
constexpr int kSumRows = 8;
template <int BM>
__global__ __launch_bounds__(256) void sum_parts_kernel(Fp8Params p) {
  const Fp8Gemm& g = p.g;
  const int n_nt = (g.N + kBN - 1) / kBN;
  const MTiles mtiles = count_tiles(g, BM);
  const int n_mt = min(p.n_mt, mtiles.total);
  const TileSplit sp = tile_split(n_nt * n_mt, (g.Kd + kBK - 1) / kBK);
  const int i = static_cast<int>(blockIdx.x) / (BM / kSumRows);
  if (i >= sp.rest) return;
  int mt, nt, e, row0, rows;
  tile_place(sp.full + i, n_nt, n_mt, &mt, &nt);
  tile_owner(g, mtiles, BM, mt, &e, &row0, &rows);
  const int r0 = static_cast<int>(blockIdx.x) % (BM / kSumRows) * kSumRows;
  const int c = static_cast<int>(threadIdx.x) % 64 * 4, n = nt * kBN + c;
  if (n >= g.N) return;
#pragma unroll
  for (int j = 0; j < kSumRows / 4; ++j) {
    const int r = r0 + j * 4 + static_cast<int>(threadIdx.x) / 64;
    if (r >= rows) return;
    const size_t step = static_cast<size_t>(sp.rest) * BM * kBN;
    const float* src = p.parts + (static_cast<size_t>(i) * BM + r) * kBN + c;
    f32x4_t v[kMaxParts];
#pragma unroll
    for (int k = 0; k < kMaxParts; ++k)
      if (k < sp.parts) v[k] = *reinterpret_cast<const f32x4_t*>(src + k * step);
#pragma unroll
    for (int k = 1; k < kMaxParts; ++k)
      if (k < sp.parts) v[0] += v[k];
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(p.out) + static_cast<size_t>(row0 + r) * g.N + n) = v[0];
  }
}

// ---------------------------------------------------------------------------- slab kernel
//
// Groups of a few rows: the weights are read once and bound the time, so
// everything is arranged for their stream. A slab is 16 RT weight rows (SwiGLU:
// 16 of W1 and the same of W3) of one expert over the whole reduction, for up
// to MC * 16 of its rows. One block per slab, KS waves, each over one part of
// the slab's stages (128 k); the parts are added in LDS in wave order.
// Per stage of a wave: non-temporal direct-to-LDS loads of the weights, each
// covering 8 rows with 8 lanes per 128-byte line, the grouped rows the same
// way, and a byte per lane for the scales (lanes 0 .. 31: of the grouped rows,
// lanes 32 and 33: of the matrices). No load of the loop writes a register, so
// no compiler-inserted wait drains the two-stage ring. Stages past the wave's
// last issue the same loads at offsets past the end, so every stage waits for
// the same count.
// v_mfma_scale_f32_16x16x128_f8f6f4, weights as the M operand: lane (a = l / 16,
// b = l % 16) reads chunks 2 a and 2 a + 1 of weight row b and of grouped row b.
template <int MODE, int MC, int RT, int KS>
__global__ __launch_bounds__(64 * KS) void gemm_fp8_slab_kernel(Fp8Params p) {
  constexpr int NMAT = MODE == F_SWIGLU ? 2 : 1;
  constexpr int ROWS = 16 * RT;                      // weight rows of a slab
  constexpr int WSLOT = NMAT * ROWS * kCH;           // u32x4 of weights per ring stage
  constexpr int XSLOT = MC * 16 * kCH;               // of grouped rows
  constexpr int SLOT = WSLOT + XSLOT + 16;           // + one dword per lane of scales
  constexpr int L = 2 * NMAT * RT + 2 * MC + 1;      // loads per stage
  static_assert(NMAT * RT * MC * 64 <= SLOT, "the parts meet in a ring slot");
  // one array per ring slot, so that reads of one are known not to alias the loads in flight into the other
  __shared__ u32x4_t R0[KS * SLOT], R1[KS * SLOT];
  const Fp8Gemm& g = p.g;
  const int lane = threadIdx.x % 64;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int la = lane / 16, lb = lane % 16;
  const int N = g.N, Kd = g.Kd;
  const int KB = (Kd + kBK - 1) / kBK, NB = (N + kBK - 1) / kBK;
  const int nsl = (N + ROWS - 1) / ROWS;

  const MTiles mtiles = count_tiles(g, MC * 16);
  const int mt = static_cast<int>(blockIdx.x) / nsl;
  if (mt >= mtiles.total) return;
  const int n0 = (static_cast<int>(blockIdx.x) - mt * nsl) * ROWS;
  int e, row0, rows;
  tile_owner(g, mtiles, MC * 16, mt, &e, &row0, &rows);
  // this wave's stages
  const int per = (KB + KS - 1) / KS;
  const int kb0 = min(KB, w * per);
  const int nks = min(KB, kb0 + per) - kb0;

  // Per-lane offsets. Instruction j covers rows 8 j .. 8 j + 7 of either
  // operand: lane l reads row 8 j + l / 8, physical chunk l % 8, the logical
  // chunk (l % 8) ^ key(row). Rows past the end get an offset past the buffer.
  const uint32_t w_bytes = static_cast<uint32_t>(N) * static_cast<uint32_t>(Kd);
  const uint32_t x_bytes = static_cast<uint32_t>(g.x_rows) * static_cast<uint32_t>(Kd);
  const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(g.x, x_bytes);
  __amdgpu_buffer_rsrc_t rw[NMAT];
  rw[0] = buffer_rsrc(g.W + static_cast<size_t>(e) * N * Kd, w_bytes);
  if constexpr (NMAT == 2) rw[NMAT - 1] = buffer_rsrc(g.W3 + static_cast<size_t>(e) * N * Kd, w_bytes);
  auto x_row = [&](int r) {  // row of x of the slab's row r
    const int s = row0 + min(r, rows - 1);
    return g.rows != nullptr ? min(max(g.rows[s], 0), g.x_rows - 1) : s;
  };
  auto chunk_k = [&](int j) { return ((lane % 8) ^ swz_key(8 * j + lane / 8)) * 16; };
  uint32_t wvo[2 * RT], xvo[2 * MC];
#pragma unroll
  for (int j = 0; j < 2 * RT; ++j) {
    const int n = n0 + 8 * j + lane / 8;
    wvo[j] = n < N ? static_cast<uint32_t>(n) * static_cast<uint32_t>(Kd) + static_cast<uint32_t>(chunk_k(j)) : w_bytes;
  }
#pragma unroll
  for (int j = 0; j < 2 * MC; ++j) {
    const int r = 8 * j + lane / 8;
    const int xr = x_row(r);
    xvo[j] = r < rows ? static_cast<uint32_t>(xr) * static_cast<uint32_t>(Kd) + static_cast<uint32_t>(chunk_k(j)) : x_bytes;
  }
  // this lane's scale byte at block 0
  const uint8_t* sp = lane < 32 ? g.xs + static_cast<size_t>(x_row(lane % (MC * 16))) * KB
                                : (NMAT == 2 && lane % 2 ? g.W3s : g.Ws) + (static_cast<size_t>(e) * NB + n0 / kBK) * KB;

  // The loads of this wave's stage i into a ring slot. (Conditions combine
  // with &: short-circuit forms became branches, each with its own load.)
  auto issue = [&](int i, u32x4_t* slots) {
    // the slot's last reads are done (their MFMAs may still be on the way)
    __builtin_amdgcn_s_waitcnt(kLgkm0);
    asm volatile("" ::: "memory");
    const bool live = i < nks;
    const int kb = kb0 + i, k0 = kb * kBK;
    u32x4_t* base = slots + w * SLOT;
#pragma unroll
    for (int m = 0; m < NMAT; ++m)
#pragma unroll
      for (int j = 0; j < 2 * RT; ++j) {
        const bool ok = live & (wvo[j] < w_bytes) & (k0 + chunk_k(j) < Kd);
        lds_load<16, 2>(rw[m], ok ? wvo[j] + k0 : w_bytes, 0, base + m * ROWS * kCH + j * 64);
      }
#pragma unroll
    for (int j = 0; j < 2 * MC; ++j) {
      const bool ok = live & (xvo[j] < x_bytes) & (k0 + chunk_k(j) < Kd);
      lds_load<16>(rx, ok ? xvo[j] + k0 : x_bytes, 0, base + WSLOT + j * 64);
    }
    // the scale byte of this block (past the last one: the last one's)
    typedef __attribute__((address_space(1))) void global_void;
    typedef __attribute__((address_space(3))) void lds_void;
    __builtin_amdgcn_global_load_lds((global_void*)(sp + min(kb, KB - 1)), (lds_void*)(base + WSLOT + XSLOT), 1, 0, 0);
  };

  f32x4_t acc[NMAT][RT][MC];
#pragma unroll
  for (int m = 0; m < NMAT; ++m)
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int c = 0; c < MC; ++c) acc[m][t][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const u32x4_t* slots) {
    const u32x4_t* base = slots + w * SLOT;
    const uint8_t* sc = reinterpret_cast<const uint8_t*>(base + WSLOT + XSLOT);
    const int c0 = swz(lb, 2 * la), c1 = swz(lb, 2 * la + 1);  // (rows 16 apart share their key)
    i32x8_t xf[MC];
    int sx[MC];
#pragma unroll
    for (int c = 0; c < MC; ++c) {
      const u32x4_t* xb = base + WSLOT + c * 16 * kCH;
      xf[c] = join(xb[c0], xb[c1]);
      sx[c] = sc[(c * 16 + lb) * 4];
    }
#pragma unroll
    for (int m = 0; m < NMAT; ++m) {
      const int sw = sc[(32 + m) * 4];
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const u32x4_t* wb = base + (m * RT + t) * 16 * kCH;
        const i32x8_t wf = join(wb[c0], wb[c1]);
#pragma unroll
        for (int c = 0; c < MC; ++c)
          acc[m][t][c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf, xf[c], acc[m][t][c], 0, 0, 0, sw, 0, sx[c]);
      }
    }
  };

  issue(0, R0);
  for (int i = 0; i < nks; i += 2) {
    issue(i + 1, R1);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(L));
    asm volatile("" ::: "memory");
    compute(R0);
    if (i + 1 < nks) {
      issue(i + 2, R0);
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(L));
      asm volatile("" ::: "memory");
      compute(R1);
    }
  }
  __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(0));  // no load may land in LDS below
  asm volatile("" ::: "memory");
  // the parts meet in this wave's own ring slot, which nothing reads or fills any more
  f32x4_t* part = reinterpret_cast<f32x4_t*>(R0 + w * SLOT);
#pragma unroll
  for (int m = 0; m < NMAT; ++m)
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int c = 0; c < MC; ++c) part[((m * RT + t) * MC + c) * 64 + lane] = acc[m][t][c];
  __syncthreads();
  if (w > 0) return;
#pragma unroll
  for (int v = 1; v < KS; ++v) {
    const f32x4_t* o = reinterpret_cast<const f32x4_t*>(R0 + v * SLOT);
#pragma unroll
    for (int m = 0; m < NMAT; ++m)
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int c = 0; c < MC; ++c) acc[m][t][c] += o[((m * RT + t) * MC + c) * 64 + lane];
  }

  // lane l holds grouped row c * 16 + l % 16 and weight rows t * 16 + 4 (l / 16) + i, i = 0 .. 3
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int n = n0 + t * 16 + la * 4;
    if (n >= N) continue;  // N % 16 == 0: four columns are all in or all out
    f32x4_t b = {0.f, 0.f, 0.f, 0.f};
    if (g.bias != nullptr) b = load_bias(g, e, n);
#pragma unroll
    for (int c = 0; c < MC; ++c) {
      const int r = c * 16 + lb;
      if (r >= rows) continue;
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = acc[0][t][c][i] + b[i];
        if (MODE == F_SWIGLU) v[i] = silu(v[i]) * acc[NMAT - 1][t][c][i];
        if (MODE == F_GELU) v[i] = gelu(v[i]);
      }
      const size_t o = static_cast<size_t>(row0 + r) * N + n;
      if (MODE == F_BF16)
        store_global(static_cast<bf16_t*>(p.out) + o, u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])});
      else
        store_global(static_cast<float*>(p.out) + o, f32x4_t{v[0], v[1], v[2], v[3]});
    }
  }
}

// Measured at 16 rows (470 MB of weights [8][14336][4096], and the decode layer's first product, twice that): four waves
// per slab 68 and 141 us, 6.9 and 6.7 TB/s, the best rate any read pattern reached on this card, so the weights' stream
// is the bound; one wave walking several slabs in turn 90 and 168 us (rows of a power-of-two length: waves at
// the same k load the same memory channels; parts of the reduction spread them); two waves 73 and 139, five or more (fewer
// blocks per CU) 87 and 171; 32 weight rows per slab instead of 16 68 against 78 (half the re-reads of the grouped rows),
// but 64 (SwiGLU with 32 of each matrix) 158 against 141; rings of three stages 116 (compiler-inserted waits).
constexpr int kSlabWaves = 4;
template <int MODE, int MC>
hipError_t launch_slab(const Fp8Gemm& g, void* out, hipStream_t st) {
  constexpr int RT = MODE == F_SWIGLU ? 1 : 2;
  Fp8Params p{g, out, nullptr, 0, nullptr};
  const int64_t blocks = most_tiles(g, MC * 16) * ((g.N + 16 * RT - 1) / (16 * RT));
  hipLaunchKernelGGL((gemm_fp8_slab_kernel<MODE, MC, RT, kSlabWaves>), dim3(static_cast<unsigned>(blocks)),
                     dim3(64 * kSlabWaves), 0, st, p);
  return hipGetLastError();
}

template <int BM, int MODE>
hipError_t launch_tile(const Fp8Gemm& g, void* out, uint8_t* qs, float* parts, hipStream_t st) {
  Fp8Params p{g, out, qs, static_cast<int>(most_tiles(g, BM)), parts};
  const int ncols = MODE == F_SWIGLU ? kBN / 2 : kBN;
  const size_t total = static_cast<size_t>((g.N + ncols - 1) / ncols) * p.n_mt;
  const size_t grid = (total + 7) / 8 * 8;
  if constexpr (MODE == F_F32) {
    if (parts != nullptr) {
      hipLaunchKernelGGL((gemm_fp8_tile_kernel<BM, MODE, true>), dim3(static_cast<unsigned>(grid + kCUs)), dim3(512), 0,
                         st, p);
      const hipError_t err = hipGetLastError();
      if (err != hipSuccess) return err;
      const size_t most = std::min(total, static_cast<size_t>(kCUs / 2));  // tiles that can be split
      hipLaunchKernelGGL(sum_parts_kernel<BM>, dim3(static_cast<unsigned>(most * (BM / kSumRows))), dim3(256), 0, st, p);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((gemm_fp8_tile_kernel<BM, MODE, false>), dim3(static_cast<unsigned>(grid)), dim3(512), 0, st, p);
  return hipGetLastError();
}

// Which kernel: rows of a slab (16 or 32), or 0 for tiles. No result's rows depend on it beyond the order of sums.
// Measured, us, slabs of 16 rows / of 32 / 128-row tiles, at the mean number of rows per expert:
//   8 experts, N 14336, Kd 4096:    mean 8: 74 / 83 / 114; 16: 111 / 90 / 115; 24: - / 101 / 115; 30: - / 136 / 116
//   128 experts, N 2048, Kd 2048:   mean 2: 80 / 103 / 96; 8: 100 / 125 / 103; 16: - / 136 / 105
//   128 experts, N 2048, Kd 512:    mean 2: 43 / 62 / 36;  64 experts, N 1024, Kd 256: mean 4: 12 / 17 / 8
//   24 experts, N 1024, Kd 1024 (96 tiles): mean 4: 8.2 / 11.7 / 9.5; 8, N 1024, Kd 512: mean 24: - / 5.5 / 6.5
// The tiles keep one block per CU busy and stream 5.1 TB/s once there are a few hundred; slabs reach 6.9 over a long
// reduction, but their start and end cost more than a short one.
int slab_rows(const Fp8Gemm& g) {
  const bool few_tiles = static_cast<int64_t>(g.E) * ((g.N + kBN - 1) / kBN) <= 256;
  const int64_t S = g.S, E = g.E;
  if (S <= 12 * E || g.max_rows <= 16) return few_tiles || g.Kd >= 2048 ? 16 : 0;
  if (S <= 24 * E || g.max_rows <= 32) return few_tiles || g.Kd >= 4096 ? 32 : 0;
  return 0;
}

// Reductions from which the last tiles are split. Measured, layer of 8 experts of d 4096, whole / split: width 14336, 4096
// tokens (576 tiles, the last 64 in 4 parts): second product 565 / 471 us, 17 of them the sum; 256 and 128 tokens (about 144
// and 128 tiles): 120 / 102 and 109 / 97; width 4096, layer of 4096, 1024 and 256 tokens: 500 / 491, 195 / 206, 132 / 132.
constexpr int kSplitKd = 8192;

// 256-row tiles, or 128: by the rounds of tiles on the CUs that groups of about the mean size take, a round of 256 rows
// costing 1.6 of 128 (measured 1.3 .. 1.75). us, 128 / 256 rows, and the rounds: 8 experts, N 14336, Kd 4096, 256 rows each
// 176 / 176 (5 / 3); 512: 291 / 272 (8 / 5); 1024: 530 / 461 (15 / 8). N 4096, Kd 14336, 512 rows: 327 / 350 (3 / 2); 1024:
// 528 / 503 (5 / 3). N 2048, Kd 2048, 512 rows: 33 / 27 (2 / 1); 1024: 49 / 52 (3 / 2); 2048: 84 / 80 (5 / 3). One expert,
// N 4096, Kd 4096, 2048 rows: 34 / 44 (1 / 1); 4096: 64 / 56 (2 / 1). 256 experts of 32 rows, N 2048: 81 / 92 (6 / 5).
// Never below 256 rows per expert: 64 experts of 128, SwiGLU, N 1376, Kd 4096: 209 / 243 (5 / 3).
template <int MODE>
bool use_256(const Fp8Gemm& g) {
  const int64_t cols = MODE == F_SWIGLU ? kBN / 2 : kBN, n_nt = (g.N + cols - 1) / cols;
  auto rounds = [&](int bm) { return ((g.S / bm + g.E / 2) * n_nt + kCUs - 1) / kCUs; };
  return g.S / g.E >= 256 && 8 * rounds(256) <= 5 * rounds(128);
}

template <int MODE>
hipError_t launch(const Fp8Gemm& g, void* out, uint8_t* qs, float* parts, hipStream_t st) {
  return use_256<MODE>(g) ? launch_tile<256, MODE>(g, out, qs, parts, st) : launch_tile<128, MODE>(g, out, qs, parts, st);
}
template <int MODE>
hipError_t launch_slabs(const Fp8Gemm& g, void* out, hipStream_t st) {
  return slab_rows(g) == 16 ? launch_slab<MODE, 1>(g, out, st) : launch_slab<MODE, 2>(g, out, st);
}

}  // namespace

size_t fp8_parts_bytes(const Fp8Gemm& g) {
  if (slab_rows(g) > 0 || g.Kd < kSplitKd) return 0;
  return static_cast<size_t>(kCUs) * (use_256<F_F32>(g) ? 256 : 128) * kBN * 4;
}

hipError_t launch_gemm_fp8(const Fp8Gemm& g, int out_type, void* out, void* parts, hipStream_t st) {
  if (slab_rows(g) > 0) return out_type == FP8_OUT_F32 ? launch_slabs<F_F32>(g, out, st) : launch_slabs<F_BF16>(g, out, st);
  if (out_type != FP8_OUT_F32) return launch<F_BF16>(g, out, nullptr, nullptr, st);
  return launch<F_F32>(g, out, nullptr, fp8_parts_bytes(g) > 0 ? static_cast<float*>(parts) : nullptr, st);
}

size_t fp8_act_tmp_bytes(const Fp8Gemm& g) { return slab_rows(g) > 0 ? static_cast<size_t>(g.S) * g.N * 4 : 0; }

hipError_t launch_gemm_fp8_act(const Fp8Gemm& g, int act, uint8_t* q, uint8_t* qs, void* tmp, hipStream_t st) {
  const bool swiglu = act == MOE_ACT_SWIGLU;
  if (slab_rows(g) == 0) return swiglu ? launch<F_SWIGLU>(g, q, qs, nullptr, st) : launch<F_GELU>(g, q, qs, nullptr, st);
  // A slab holds 16 columns and a scale needs 128: the activations go through
  // float32 rows and the quantiser (a few rows; rows that no expert holds are
  // converted too, whatever they are, and read by nothing).
  const hipError_t err = swiglu ? launch_slabs<F_SWIGLU>(g, tmp, st) : launch_slabs<F_GELU>(g, tmp, st);
  if (err != hipSuccess) return err;
  return launch_quantize_fp8(tmp, false, 1, g.S, g.N, 1, q, qs, st);
}

}  // namespace moe
