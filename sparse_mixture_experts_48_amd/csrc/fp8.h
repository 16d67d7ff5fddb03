// Launch interface of the grouped router, the grouping without copied rows,
// the 8-bit quantiser and the block-scaled 8-bit products.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int kFp8Block = 128;      // values that share a scale, along the reduction (and rows of a weight)
constexpr int kMaxExperts = 512;    // of the grouped router, the grouping and the 8-bit products
constexpr int kMaxGroups = 32;
constexpr int32_t kNoExpert = 0x7fffffff;  // the id of a choice that no expert was left for

struct GroupedRouteArgs {
  const void* logits;  // [T][E], bfloat16 or float32
  bool bf16;
  const float* bias;   // [E] or null
  int T, E, K, groups, top_groups, group_top;
  bool sigmoid, renorm;
  float scale;
};
hipError_t launch_route_grouped(const GroupedRouteArgs& a, int32_t* topk_idx, float* topk_gate, hipStream_t st);
hipError_t launch_route_grouped_backward(const GroupedRouteArgs& a, const int32_t* topk_idx, const float* dgate,
                                         void* dlogits, hipStream_t st);

// x [rows][cols] to e4m3 with a power-of-two scale (E8M0) per block of 1 x 128.
struct QuantRows {
  const void* x;
  int64_t rows, cols;
  uint8_t *q, *scale;
};

// Grouping: blocks of group_chunk(S) slots; blk_hist holds group_blocks(S) rows of E counts. quant: nullable, rows
// (bfloat16 or float32) that the first launch quantises beside the grouping.
int group_blocks(int64_t S);
hipError_t launch_group(const int32_t* topk_idx, int S, int E, int K, int32_t* counts, int32_t* offsets,
                        int32_t* slot_token, int32_t* token_slot, int32_t* blk_hist, const QuantRows* quant, bool quant_bf16,
                        hipStream_t st);

// mats matrices [rows][cols] to e4m3 with a power-of-two scale (E8M0) per block of br x 128 (br = 1 or 128).
hipError_t launch_quantize_fp8(const void* x, bool bf16, int64_t mats, int64_t rows, int64_t cols, int br, uint8_t* q,
                               uint8_t* scale, hipStream_t st);

// Grouped products of 8-bit operands.
enum { FP8_OUT_F32 = 0, FP8_OUT_BF16 = 1 };
struct Fp8Gemm {
  const uint8_t* x;        // e4m3 [x_rows][Kd]
  const uint8_t* xs;       // E8M0 [x_rows][ceil(Kd / 128)]
  const int32_t* rows;     // nullable: grouped row s is row rows[s] of x
  const int32_t* offsets;  // [E + 1]; null: E = 1, every row
  const uint8_t* W;        // e4m3 [E][N][Kd]
  const uint8_t* Ws;       // E8M0 [E][ceil(N / 128)][ceil(Kd / 128)]
  const uint8_t* W3;       // SwiGLU: the second matrix and its scales
  const uint8_t* W3s;
  const void* bias;        // [E][N] or null
  bool bias_bf16;
  int S, x_rows, E, N, Kd;
  int max_rows;            // rows that the largest group is expected to have: may pick the kernel (and the order of the sums)
};
// out [S][N] float32 or bfloat16. parts: fp8_parts_bytes of scratch for tiles split along the reduction (float32
// output), or null for none.
size_t fp8_parts_bytes(const Fp8Gemm& g);
hipError_t launch_gemm_fp8(const Fp8Gemm& g, int out_type, void* out, void* parts, hipStream_t st);
// The first expert product with its activation: a = act(.) of every grouped row as e4m3 with a scale per 128
// columns: q [S][N], qs [S][ceil(N / 128)]. act: moe_act. tmp: fp8_act_tmp_bytes (of S, E, N, Kd and max_rows) of scratch.
size_t fp8_act_tmp_bytes(const Fp8Gemm& g);
hipError_t launch_gemm_fp8_act(const Fp8Gemm& g, int act, uint8_t* q, uint8_t* qs, void* tmp, hipStream_t st);

}  // namespace moe
