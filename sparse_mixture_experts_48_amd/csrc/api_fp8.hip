// C-ABI of the grouped router, the grouping without copied rows, the 8-bit
// quantiser, the block-scaled 8-bit products and the layer built of them
// (declared in include/moe.h).
#include <algorithm>
#include <cmath>

#include "api_common.h"
#include "fp8.h"
#include "kernels.h"

namespace {

using moe::align_up;
using moe::at;
using moe::check_ptr;
using moe::check_ws;
using moe::kMaxDim;
using moe::kMaxElems;
using moe::kMaxInt;

constexpr int64_t kMaxLaunch = (int64_t{1} << 32) - 256;  // threads of a launch at most

int64_t blocks_of(int64_t n) { return (n + moe::kFp8Block - 1) / moe::kFp8Block; }

int check_dtype(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 ? MOE_OK : MOE_ERR_UNSUPPORTED; }

int check_choices(int64_t T, int64_t E, int64_t K) {
  if (T < 0 || E < 1 || K < 1) return MOE_ERR_SHAPE;
  if (E > moe::kMaxExperts || K > 8 || T > kMaxInt / K) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_router(const moe_router_desc* r) {
  if (r == nullptr) return MOE_ERR_NULL;
  if (r->T < 0 || r->E < 1 || r->K < 1 || r->groups < 1 || r->E % r->groups != 0) return MOE_ERR_SHAPE;
  if (r->top_groups < 1 || r->top_groups > r->groups) return MOE_ERR_SHAPE;
  if (r->K > r->top_groups * (r->E / r->groups) || !std::isfinite(r->scale)) return MOE_ERR_SHAPE;
  if (r->groups > moe::kMaxGroups) return MOE_ERR_UNSUPPORTED;
  if (r->group_top != 1 && r->group_top != 2) return MOE_ERR_UNSUPPORTED;
  if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) return MOE_ERR_UNSUPPORTED;
  if (r->renorm != 0 && r->renorm != 1) return MOE_ERR_UNSUPPORTED;
  MOE_CHECK(check_choices(r->T, r->E, r->K));
  if (r->T > kMaxLaunch / 16) return MOE_ERR_UNSUPPORTED;  // 16 threads per token
  return r->T > 0 && r->T > kMaxElems / r->E ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe::GroupedRouteArgs route_args(const moe_router_desc& r, const void* logits, int dtype, const float* bias) {
  return moe::GroupedRouteArgs{logits, dtype == MOE_BF16, bias, static_cast<int>(r.T), static_cast<int>(r.E),
                               static_cast<int>(r.K), static_cast<int>(r.groups), static_cast<int>(r.top_groups),
                               r.group_top, r.score == MOE_SCORE_SIGMOID, r.renorm != 0, r.scale};
}

size_t group_ws(int64_t T, int64_t E, int64_t K) {
  const int64_t S = T * K;
  return S > 0 ? align_up(static_cast<size_t>(moe::group_blocks(S)) * E * 4) : 0;
}

// A product's operands: S grouped rows of Kd values against experts' [N][Kd].
int check_product(int64_t S, int64_t x_rows, int64_t E, int64_t N, int64_t Kd) {
  if (S < 0 || x_rows < 0 || E < 1 || N < 1 || Kd < 1) return MOE_ERR_SHAPE;
  if (E > moe::kMaxExperts || N % 16 != 0 || Kd % 16 != 0 || N > kMaxDim || Kd > kMaxDim) return MOE_ERR_UNSUPPORTED;
  if (S > kMaxInt - 65536 || N > kMaxElems / Kd) return MOE_ERR_UNSUPPORTED;
  if ((x_rows > 0 && x_rows > kMaxElems / Kd) || (S > 0 && S > kMaxElems / N)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Shapes of the 8-bit layer: those of a moe_desc, up to 512 experts, dropless.
int check_fp8_desc(const moe_desc* d) {
  if (d == nullptr) return MOE_ERR_NULL;
  if (d->T < 0 || d->d < 1 || d->width < 1 || d->E < 1 || d->K < 1 || d->K > d->E || d->capacity < 0)
    return MOE_ERR_SHAPE;
  if (d->act != MOE_ACT_GELU && d->act != MOE_ACT_SWIGLU) return MOE_ERR_UNSUPPORTED;
  if (d->capacity != 0 || d->bias_mode != MOE_BIAS_LOGITS) return MOE_ERR_UNSUPPORTED;
  MOE_CHECK(check_dtype(d->dtype));
  MOE_CHECK(check_choices(d->T, d->E, d->K));
  MOE_CHECK(check_product(d->T * d->K, d->T * d->K, d->E, d->width, d->d));
  return check_product(d->T * d->K, d->T * d->K, d->E, d->d, d->width);
}

struct Fp8Plan {
  size_t hq, hs, aq, as, tmp, parts;  // 8-bit tokens, hidden activations, sums of split tiles
  size_t topk_idx, topk_gate, counts, offsets, slot_token, token_slot, group, o_perm;  // the layer's routing and rows
  size_t total;
};

Fp8Plan make_fp8_plan(const moe_desc& d) {
  Fp8Plan p{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align_up(bytes);
    return o;
  };
  const size_t T = d.T, S = static_cast<size_t>(d.T) * d.K;
  p.aq = take(S * d.width);
  p.as = take(S * blocks_of(d.width));
  moe::Fp8Gemm g{};
  g.S = static_cast<int>(S);
  g.E = static_cast<int>(d.E);
  g.N = static_cast<int>(d.width);
  g.Kd = static_cast<int>(d.d);
  g.max_rows = static_cast<int>(d.T);
  p.tmp = take(moe::fp8_act_tmp_bytes(g));
  g.N = static_cast<int>(d.d);
  g.Kd = static_cast<int>(d.width);
  p.parts = take(moe::fp8_parts_bytes(g));
  p.hq = take(T * d.d);
  p.hs = take(T * blocks_of(d.d));
  p.topk_idx = take(S * 4);
  p.topk_gate = take(S * 4);
  p.counts = take(d.E * 4);
  p.offsets = take((d.E + 1) * 4);
  p.slot_token = take(S * 4);
  p.token_slot = take(S * 4);
  p.group = take(group_ws(d.T, d.E, d.K));
  p.o_perm = take(S * d.d * 4);
  p.total = off;
  return p;
}

struct Fp8Weights {
  const void *W1, *s1, *b1, *W3, *s3, *W2, *s2, *b2;
};

int check_weights(const moe_desc& d, const Fp8Weights& w) {
  MOE_CHECK(check_ptr(w.W1, true));
  MOE_CHECK(check_ptr(w.s1, true));
  MOE_CHECK(check_ptr(w.W2, true));
  MOE_CHECK(check_ptr(w.s2, true));
  if (d.act == MOE_ACT_SWIGLU) {
    MOE_CHECK(check_ptr(w.W3, true));
    MOE_CHECK(check_ptr(w.s3, true));
    if (w.b1 != nullptr || w.b2 != nullptr) return MOE_ERR_UNSUPPORTED;
  }
  MOE_CHECK(check_ptr(w.b1, false));
  return check_ptr(w.b2, false);
}

// Both products of the expert MLP on the rows of x (through rows unless null).
int enqueue_ffn(const moe_desc& d, const Fp8Plan& pl, const void* x, const void* xs, const int32_t* rows, int x_rows,
                const int32_t* offsets, const Fp8Weights& w, float* o_perm, void* ws, hipStream_t st) {
  const int S = static_cast<int>(d.T * d.K);
  moe::Fp8Gemm g{};
  g.x = static_cast<const uint8_t*>(x);
  g.xs = static_cast<const uint8_t*>(xs);
  g.rows = rows;
  g.offsets = offsets;
  g.W = static_cast<const uint8_t*>(w.W1);
  g.Ws = static_cast<const uint8_t*>(w.s1);
  g.W3 = static_cast<const uint8_t*>(w.W3);
  g.W3s = static_cast<const uint8_t*>(w.s3);
  g.bias = w.b1;
  g.bias_bf16 = d.dtype == MOE_BF16;
  g.S = S;
  g.x_rows = x_rows;
  g.E = static_cast<int>(d.E);
  g.N = static_cast<int>(d.width);
  g.Kd = static_cast<int>(d.d);
  g.max_rows = static_cast<int>(d.T);  // a token chooses distinct experts
  uint8_t* aq = at<uint8_t>(ws, pl.aq);
  uint8_t* as = at<uint8_t>(ws, pl.as);
  MOE_LAUNCH(MOE_K_GEMM1, st, moe::launch_gemm_fp8_act(g, d.act, aq, as, at<char>(ws, pl.tmp), st));
  g.x = aq;
  g.xs = as;
  g.rows = nullptr;
  g.W = static_cast<const uint8_t*>(w.W2);
  g.Ws = static_cast<const uint8_t*>(w.s2);
  g.W3 = g.W3s = nullptr;
  g.bias = w.b2;
  g.x_rows = S;
  g.N = static_cast<int>(d.d);
  g.Kd = static_cast<int>(d.width);
  MOE_LAUNCH(MOE_K_GEMM2, st, moe::launch_gemm_fp8(g, moe::FP8_OUT_F32, o_perm, at<char>(ws, pl.parts), st));
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_route_grouped(const moe_router_desc* desc, const void* logits, int logits_dtype, const float* bias,
                      int32_t* topk_idx, float* topk_gate, void* stream) {
  MOE_CHECK(check_router(desc));
  MOE_CHECK(check_dtype(logits_dtype));
  const bool any = desc->T > 0;
  MOE_CHECK(check_ptr(logits, any));
  MOE_CHECK(check_ptr(bias, false));
  MOE_CHECK(check_ptr(topk_idx, any));
  MOE_CHECK(check_ptr(topk_gate, any));
  if (!any) return MOE_OK;
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_LAUNCH(MOE_K_ROUTE, st,
             moe::launch_route_grouped(route_args(*desc, logits, logits_dtype, bias), topk_idx, topk_gate, st));
  return MOE_OK;
}

int moe_route_grouped_backward(const moe_router_desc* desc, const void* logits, int logits_dtype,
                               const int32_t* topk_idx, const float* dgate, void* dlogits, void* stream) {
  MOE_CHECK(check_router(desc));
  MOE_CHECK(check_dtype(logits_dtype));
  const bool any = desc->T > 0;
  MOE_CHECK(check_ptr(logits, any));
  MOE_CHECK(check_ptr(topk_idx, any));
  MOE_CHECK(check_ptr(dgate, any));
  MOE_CHECK(check_ptr(dlogits, any));
  if (!any) return MOE_OK;
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_LAUNCH(MOE_K_BWD, st,
             moe::launch_route_grouped_backward(route_args(*desc, logits, logits_dtype, nullptr), topk_idx, dgate,
                                                dlogits, st));
  return MOE_OK;
}

int moe_group_workspace_size(int64_t T, int64_t E, int64_t K, size_t* bytes) {
  if (bytes == nullptr) return MOE_ERR_NULL;
  MOE_CHECK(check_choices(T, E, K));
  *bytes = group_ws(T, E, K);
  return MOE_OK;
}

int moe_group(int64_t T, int64_t E, int64_t K, const int32_t* topk_idx, int32_t* expert_counts,
              int32_t* expert_offsets, int32_t* slot_token, int32_t* token_slot, void* ws, size_t ws_bytes,
              void* stream) {
  MOE_CHECK(check_choices(T, E, K));
  const bool any = T > 0;
  MOE_CHECK(check_ptr(topk_idx, any));
  MOE_CHECK(check_ptr(expert_counts, true));
  MOE_CHECK(check_ptr(expert_offsets, true));
  MOE_CHECK(check_ptr(slot_token, any));
  MOE_CHECK(check_ptr(token_slot, any));
  MOE_CHECK(check_ws(group_ws(T, E, K), ws, ws_bytes));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_LAUNCH(MOE_K_PERMUTE, st,
             moe::launch_group(topk_idx, static_cast<int>(T * K), static_cast<int>(E), static_cast<int>(K),
                               expert_counts, expert_offsets, slot_token, token_slot, at<int32_t>(ws, 0), nullptr, false,
                               st));
  return MOE_OK;
}

int moe_quantize_fp8(const void* x, int dtype, int64_t mats, int64_t rows, int64_t cols, int block_rows, void* q,
                     void* scale, void* stream) {
  MOE_CHECK(check_dtype(dtype));
  if (mats < 0 || rows < 0 || cols < 1) return MOE_ERR_SHAPE;
  if (block_rows != 1 && block_rows != moe::kFp8Block) return MOE_ERR_UNSUPPORTED;
  if (cols % 16 != 0 || cols > kMaxDim || mats > kMaxInt || rows > kMaxInt) return MOE_ERR_UNSUPPORTED;
  const bool any = mats > 0 && rows > 0;
  // 16 threads per block of a row's scales, 256 per block of 128 x 128
  const int64_t threads = blocks_of(cols) * (block_rows == 1 ? 16 : 256);
  if (any && mats * (block_rows == 1 ? rows : blocks_of(rows)) > kMaxLaunch / threads) return MOE_ERR_UNSUPPORTED;
  MOE_CHECK(check_ptr(x, any));
  MOE_CHECK(check_ptr(q, any));
  MOE_CHECK(check_ptr(scale, any));
  if (!any) return MOE_OK;
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_LAUNCH(MOE_K_QUANTIZE, st,
             moe::launch_quantize_fp8(x, dtype == MOE_BF16, mats, rows, cols, block_rows, static_cast<uint8_t*>(q),
                                      static_cast<uint8_t*>(scale), st));
  return MOE_OK;
}

int moe_grouped_gemm_fp8(const moe_gemm_fp8_desc* desc, const void* x, const void* x_scale, const int32_t* rows,
                         const int32_t* offsets, const void* W, const void* W_scale, const void* bias, void* out,
                         void* stream) {
  if (desc == nullptr) return MOE_ERR_NULL;
  const moe_gemm_fp8_desc& d = *desc;
  MOE_CHECK(check_product(d.S, d.x_rows, d.E, d.N, d.Kd));
  if (d.max_rows < 0) return MOE_ERR_SHAPE;
  MOE_CHECK(check_dtype(d.out_dtype));
  MOE_CHECK(check_dtype(d.bias_dtype));
  const bool any = d.S > 0;
  if (any && d.x_rows < 1) return MOE_ERR_SHAPE;
  if (rows == nullptr && d.x_rows != d.S) return MOE_ERR_SHAPE;
  if (offsets == nullptr && d.E != 1) return MOE_ERR_NULL;
  MOE_CHECK(check_ptr(x, any));
  MOE_CHECK(check_ptr(x_scale, any));
  MOE_CHECK(check_ptr(rows, false));
  MOE_CHECK(check_ptr(offsets, false));
  MOE_CHECK(check_ptr(W, true));
  MOE_CHECK(check_ptr(W_scale, true));
  MOE_CHECK(check_ptr(bias, false));
  MOE_CHECK(check_ptr(out, any));
  if (!any) return MOE_OK;
  moe::Fp8Gemm g{};
  g.x = static_cast<const uint8_t*>(x);
  g.xs = static_cast<const uint8_t*>(x_scale);
  g.rows = rows;
  g.offsets = offsets;
  g.W = static_cast<const uint8_t*>(W);
  g.Ws = static_cast<const uint8_t*>(W_scale);
  g.bias = bias;
  g.bias_bf16 = d.bias_dtype == MOE_BF16;
  g.S = static_cast<int>(d.S);
  g.x_rows = static_cast<int>(d.x_rows);
  g.E = static_cast<int>(d.E);
  g.N = static_cast<int>(d.N);
  g.Kd = static_cast<int>(d.Kd);
  g.max_rows = static_cast<int>(d.max_rows == 0 ? d.S : std::min(d.max_rows, d.S));
  hipStream_t st = static_cast<hipStream_t>(stream);
  MOE_LAUNCH(MOE_K_GEMM2, st,
             moe::launch_gemm_fp8(g, d.out_dtype == MOE_BF16 ? moe::FP8_OUT_BF16 : moe::FP8_OUT_F32, out, nullptr, st));
  return MOE_OK;
}

int moe_fp8_workspace_size(const moe_desc* desc, size_t* bytes) {
  if (bytes == nullptr) return MOE_ERR_NULL;
  MOE_CHECK(check_fp8_desc(desc));
  *bytes = make_fp8_plan(*desc).total;
  return MOE_OK;
}

int moe_expert_ffn_fp8(const moe_desc* desc, const void* x, const void* x_scale, const int32_t* rows,
                       const int32_t* expert_offsets, const void* W1, const void* W1_scale, const void* b1,
                       const void* W3, const void* W3_scale, const void* W2, const void* W2_scale, const void* b2,
                       float* o_perm, void* ws, size_t ws_bytes, void* stream) {
  MOE_CHECK(check_fp8_desc(desc));
  const moe_desc& d = *desc;
  const Fp8Plan pl = make_fp8_plan(d);
  const Fp8Weights w{W1, W1_scale, b1, W3, W3_scale, W2, W2_scale, b2};
  const bool any = d.T > 0;
  MOE_CHECK(check_ptr(x, any));
  MOE_CHECK(check_ptr(x_scale, any));
  MOE_CHECK(check_ptr(rows, false));
  MOE_CHECK(check_ptr(expert_offsets, any));
  MOE_CHECK(check_weights(d, w));
  MOE_CHECK(check_ptr(o_perm, any));
  MOE_CHECK(check_ws(pl.total, ws, ws_bytes));
  if (!any) return MOE_OK;
  return enqueue_ffn(d, pl, x, x_scale, rows, static_cast<int>(rows != nullptr ? d.T : d.T * d.K), expert_offsets, w,
                     o_perm, ws, static_cast<hipStream_t>(stream));
}

int moe_forward_fp8(const moe_desc* desc, const moe_router_desc* router, const void* h, const void* logits,
                    int logits_dtype, const float* bias, const void* W1, const void* W1_scale, const void* b1,
                    const void* W3, const void* W3_scale, const void* W2, const void* W2_scale, const void* b2, void* y,
                    int32_t* topk_idx, float* topk_gate, int32_t* expert_counts, void* ws, size_t ws_bytes,
                    void* stream) {
  MOE_CHECK(check_fp8_desc(desc));
  MOE_CHECK(check_router(router));
  MOE_CHECK(check_dtype(logits_dtype));
  const moe_desc& d = *desc;
  if (router->T != d.T || router->E != d.E || router->K != d.K) return MOE_ERR_SHAPE;
  const Fp8Plan pl = make_fp8_plan(d);
  const Fp8Weights w{W1, W1_scale, b1, W3, W3_scale, W2, W2_scale, b2};
  const bool any = d.T > 0;
  MOE_CHECK(check_ptr(h, any));
  MOE_CHECK(check_ptr(logits, any));
  MOE_CHECK(check_ptr(bias, false));
  MOE_CHECK(check_weights(d, w));
  MOE_CHECK(check_ptr(y, any));
  MOE_CHECK(check_ptr(topk_idx, false));
  MOE_CHECK(check_ptr(topk_gate, false));
  MOE_CHECK(check_ptr(expert_counts, false));
  MOE_CHECK(check_ws(pl.total, ws, ws_bytes));
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int T = static_cast<int>(d.T), E = static_cast<int>(d.E), K = static_cast<int>(d.K), S = T * K;
  int32_t* idx = topk_idx != nullptr ? topk_idx : at<int32_t>(ws, pl.topk_idx);
  float* gate = topk_gate != nullptr ? topk_gate : at<float>(ws, pl.topk_gate);
  int32_t* counts = expert_counts != nullptr ? expert_counts : at<int32_t>(ws, pl.counts);
  int32_t* offsets = at<int32_t>(ws, pl.offsets);
  int32_t* slot_token = at<int32_t>(ws, pl.slot_token);
  int32_t* token_slot = at<int32_t>(ws, pl.token_slot);
  if (any)
    MOE_LAUNCH(MOE_K_ROUTE, st,
               moe::launch_route_grouped(route_args(*router, logits, logits_dtype, bias), idx, gate, st));
  uint8_t* hq = at<uint8_t>(ws, pl.hq);
  uint8_t* hs = at<uint8_t>(ws, pl.hs);
  const moe::QuantRows quant{h, d.T, d.d, hq, hs};
  MOE_LAUNCH(MOE_K_PERMUTE, st,
             moe::launch_group(idx, S, E, K, counts, offsets, slot_token, token_slot, at<int32_t>(ws, pl.group),
                               any ? &quant : nullptr, d.dtype == MOE_BF16, st));
  if (!any) return MOE_OK;
  float* o_perm = at<float>(ws, pl.o_perm);
  MOE_CHECK(enqueue_ffn(d, pl, hq, hs, slot_token, T, offsets, w, o_perm, ws, st));
  MOE_LAUNCH(MOE_K_COMBINE, st,
             moe::launch_combine(o_perm, token_slot, gate, T, static_cast<int>(d.d), K, d.dtype == MOE_BF16, y, st));
  return MOE_OK;
}

}  // extern "C"
