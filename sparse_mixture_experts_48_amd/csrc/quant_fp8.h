// Device pieces of the 8-bit quantiser, shared by its own kernels, the grouping
// launch that quantises the layer's tokens and the products' epilogues.
#pragma once

#include "common.h"
#include "fp8.h"

namespace moe {

// Scale byte of a block whose largest magnitude has the bits amax (448 = 1.75 2^8).
__device__ __forceinline__ int scale_byte(uint32_t amax) {
  const int b = static_cast<int>(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(b, 0);
}
// 2^(127 - byte) for byte 0 .. 247
__device__ __forceinline__ float inverse_scale(int byte) { return __uint_as_float(static_cast<uint32_t>(254 - byte) << 23); }

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* v);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float* v) {
  const f32x4_t a = *reinterpret_cast<const f32x4_t*>(p), b = *reinterpret_cast<const f32x4_t*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
}
template <>
__device__ __forceinline__ void load8<bf16_t>(const bf16_t* p, float* v) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// bits of max |v|; a NaN does not take part (its own value stays NaN)
__device__ __forceinline__ uint32_t amax8(const float* v) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return __float_as_uint(m);
}

__device__ __forceinline__ uint2 pack8(const float* v, float f) {
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * f, v[1] * f, 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * f, v[3] * f, lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * f, v[5] * f, 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * f, v[7] * f, hi, true);
  return make_uint2(static_cast<uint32_t>(lo), static_cast<uint32_t>(hi));
}

// Rows by blocks of 1 x 128: thread i of the call takes 8 values of block i / 16 (16 lanes per block).
template <typename T>
__device__ __forceinline__ void quant_rows(const QuantRows& a, int64_t i) {
  const int64_t kb = (a.cols + kFp8Block - 1) / kFp8Block;
  const int64_t blk = i / 16;
  const int l = static_cast<int>(i % 16);
  if (blk >= a.rows * kb) return;
  const int64_t r = blk / kb, c = (blk - r * kb) * kFp8Block + l * 8;
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = 0.0f;
  if (c < a.cols) load8(static_cast<const T*>(a.x) + r * a.cols + c, v);
  uint32_t m = amax8(v);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), o)));
  const int b = scale_byte(m);
  if (c < a.cols) *reinterpret_cast<uint2*>(a.q + r * a.cols + c) = pack8(v, inverse_scale(b));
  if (l == 0) a.scale[blk] = static_cast<uint8_t>(b);
}

}  // namespace moe
