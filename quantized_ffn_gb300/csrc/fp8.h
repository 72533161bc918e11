// fp8.h -- block-scaled e4m3: conversion helpers and the launchers of
// fp8_quant.cu (quantise, dequantise) and fp8_matmul.cu (products).
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace zffn {

constexpr int kF8Block = 128;   // values that share a scale along a row

__host__ __device__ inline int64_t f8_blocks(int64_t n) { return (n + kF8Block - 1) / kF8Block; }

#ifdef __CUDACC__
// Exponent p of the block scale 2^p: the least p >= -126 with amax <= 448 * 2^p.
// 448 * 2^p = 1.75 * 2^(p+8), so p follows from amax's exponent field and from
// its mantissa's place against 1.75 (0.75 is 0x600000).  0 for amax = 0.
__device__ __forceinline__ int f8_scale_exp(float amax) {
    const uint32_t u = __float_as_uint(amax);
    if (u == 0) return 0;
    const int p = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return p < -126 ? -126 : p;
}
__device__ __forceinline__ float pow2f(int p) { return __uint_as_float((uint32_t)(p + 127) << 23); }
// |x| where it is finite, 0 for infinities and NaN (they set no scale).
__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? a : 0.0f;
}
// Two fp32 values -> two e4m3 bytes (lo in the low byte), nearest even,
// +-448 beyond the range, NaN kept.
__device__ __forceinline__ uint32_t f8x2_satfinite(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t f8x4_satfinite(float a, float b, float c, float d) {
    return f8x2_satfinite(a, b) | (f8x2_satfinite(c, d) << 16);
}
#endif

// dtype: zffn_dtype of x; block_rows 1 or 128
cudaError_t launch_fp8_quantize(int dtype, const void *x, uint8_t *q, float *scale, int64_t rows,
                                int64_t cols, int block_rows, cudaStream_t s);
cudaError_t launch_fp8_dequant(const uint8_t *q, const float *scale, float *out, int64_t rows,
                               int64_t cols, int block_rows, cudaStream_t s);

// One product: y = a . w^T (w1 == nullptr), or h = quantise(silu(a . w^T) * (a . w1^T)).
struct Fp8Args {
    const uint8_t *a;        // [M][K]
    const float *a_scale;    // [M][ceil(K/128)]
    const int32_t *offsets;  // [E + 1] rows of each expert, or nullptr (dense)
    const uint8_t *w;        // [E][N][K]
    const float *w_scale;    // [E][ceil(N/128)][ceil(K/128)]
    const uint8_t *w1;       // as w (the up projection), or nullptr
    const float *w1_scale;
    void *y;                 // [M][N] of y_dtype, or e4m3 bytes (SwiGLU)
    float *y_scale;          // SwiGLU: [M][ceil(N/128)]
    int y_dtype;             // zffn_dtype (without SwiGLU)
    int M, N, K, E;
    int *err;
    // the grid launched just before writes a and a_scale and nothing else that this
    // product reads, and it waited for the grids before it: the weights are asked
    // for before it ends
    bool early;
};
cudaError_t launch_fp8_matmul(const Fp8Args &a, cudaStream_t s);

}  // namespace zffn
