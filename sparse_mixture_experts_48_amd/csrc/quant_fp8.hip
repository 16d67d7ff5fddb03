// 8-bit quantisation: e4m3 values with one power-of-two scale for each block
// of 128 values of a row (activations) or of 128 x 128 (weights).
//
//   e = the smallest integer >= -127 with max |x| <= 448 2^e
//   q = x 2^-e rounded to the nearest e4m3 value (ties to even), scale byte e + 127 (E8M0)
//
// A power of two scales without rounding, so the result is the same in any
// arithmetic, and the scaled matrix instructions take the byte as it is.
// Memory-bound: each value is read once and written once. Measured: [8][14336][4096] bfloat16 in blocks of 128 x 128
// 262 us = 5.4 TB/s, 32768 x 4096 bfloat16 by rows 74 us = 5.4 TB/s (a copy reaches 4.9 .. 5.1), 16 x 4096 2.7 us (a
// launch). One 64-bit division per thread costs nothing beside that (one per thread block instead: 73 us).
#include "common.h"
#include "fp8.h"
#include "quant_fp8.h"

namespace moe {

namespace {

constexpr int kQT = 256;

template <typename T>
__global__ __launch_bounds__(kQT) void quant_rows_kernel(QuantRows a) {
  quant_rows<T>(a, static_cast<int64_t>(blockIdx.x) * kQT + threadIdx.x);
}

// One block per 128 x 128 values: 16 lanes across a row, 16 rows at a time, all
// 64 values of a thread in registers between the maximum and the conversion.
template <typename T>
__global__ __launch_bounds__(kQT) void quant_tiles_kernel(const T* __restrict__ x, int64_t rows, int64_t cols,
                                                          uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
  __shared__ uint32_t wm[kQT / 64];
  const int64_t rb = (rows + kFp8Block - 1) / kFp8Block, kb = (cols + kFp8Block - 1) / kFp8Block;
  const int64_t blk = blockIdx.x;
  const int64_t mat = blk / (rb * kb), in = blk - mat * rb * kb;
  const int64_t r0 = in / kb * kFp8Block, c = in % kb * kFp8Block + threadIdx.x % 16 * 8;
  x += mat * rows * cols;
  q += mat * rows * cols;
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + i * 16 + threadIdx.x / 16;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    if (r < rows && c < cols) load8(x + r * cols + c, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, amax8(v[i]));
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), o)));
  if (threadIdx.x % 64 == 0) wm[threadIdx.x / 64] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQT / 64; ++w) m = max(m, wm[w]);
  const int b = scale_byte(m);
  const float f = inverse_scale(b);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + i * 16 + threadIdx.x / 16;
    if (r < rows && c < cols) *reinterpret_cast<uint2*>(q + r * cols + c) = pack8(v[i], f);
  }
  if (threadIdx.x == 0) scale[blk] = static_cast<uint8_t>(b);
}

template <typename T>
hipError_t launch(const T* x, int64_t mats, int64_t rows, int64_t cols, int br, uint8_t* q, uint8_t* scale,
                  hipStream_t st) {
  const int64_t kb = (cols + kFp8Block - 1) / kFp8Block;
  if (br == 1) {
    const int64_t blocks = (mats * rows * kb * 16 + kQT - 1) / kQT;
    hipLaunchKernelGGL(quant_rows_kernel<T>, dim3(static_cast<unsigned>(blocks)), dim3(kQT), 0, st,
                       QuantRows{x, mats * rows, cols, q, scale});
  } else {
    const int64_t blocks = mats * ((rows + kFp8Block - 1) / kFp8Block) * kb;
    hipLaunchKernelGGL(quant_tiles_kernel<T>, dim3(static_cast<unsigned>(blocks)), dim3(kQT), 0, st, x, rows, cols, q,
                       scale);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_fp8(const void* x, bool bf16, int64_t mats, int64_t rows, int64_t cols, int br, uint8_t* q,
                               uint8_t* scale, hipStream_t st) {
  return bf16 ? launch(static_cast<const bf16_t*>(x), mats, rows, cols, br, q, scale, st)
              : launch(static_cast<const float*>(x), mats, rows, cols, br, q, scale, st);
}

}  // namespace moe
