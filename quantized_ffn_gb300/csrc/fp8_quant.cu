// fp8_quant.cu -- e4m3 with a power-of-two scale for each block of 128 columns
// of a row (activations) or each 128 x 128 block (weights), and back.
//
//   s = the least 2^p with max|x| <= 448 s,   q = e4m3(x / s)
//
// A power of two loses nothing against max|x| / 448: e4m3 has the same three
// mantissa bits in every binade, so only values below 2^-9 of the block's
// largest (subnormals) see another step, and x / s is exact, so that a value is
// rounded once and the result does not depend on how the division is done.
#include "fp8.h"

#include "zffn_internal.cuh"

namespace zffn {

namespace {

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// Eight consecutive values as fp32, by 16-byte loads.
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 f = __ldg(reinterpret_cast<const float4 *>(p) + i);
        v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
    }
}

constexpr int kQuantThreads = 256;

// 1 x 128 blocks: 16 lanes per block, 8 columns per lane.  VEC: 16-byte loads
// and 8-byte stores (rows of 16-byte multiples from 16-byte aligned pointers);
// otherwise element by element.  Bound by HBM.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kQuantThreads)
    fp8_quantize_rows_kernel(const T *__restrict__ x, uint8_t *__restrict__ q, float *__restrict__ scale,
                             int64_t rows, int cols, int nb) {
    const int sub = threadIdx.x & 15;
    const int64_t unit = (int64_t)blockIdx.x * (kQuantThreads / 16) + (threadIdx.x >> 4);
    const int64_t row = unit / nb;
    const int b = (int)(unit - row * nb);
    const bool live = row < rows;
    const int c0 = b * kF8Block + sub * 8;
    const T *px = x + (live ? row : 0) * cols;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (live) {
        if (VEC) {
            if (c0 < cols) load8(px + c0, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c0 + i < cols) v[i] = to_f32(px[c0 + i]);
        }
    }
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, finite_abs(v[i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (!live) return;
    const int p = f8_scale_exp(top);
    const float inv = pow2f(-p);
    const uint32_t lo = f8x4_satfinite(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    const uint32_t hi = f8x4_satfinite(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    uint8_t *pq = q + row * cols;
    if (VEC) {
        if (c0 < cols) *reinterpret_cast<uint2 *>(pq + c0) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c0 + i < cols) pq[c0 + i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
    if (sub == 0) scale[row * nb + b] = pow2f(p);
}

// 128 x 128 blocks: one thread block each; two passes over the block (the
// second from L1/L2), the maximum of the first between them.  Weights are
// quantised once, so this kernel is plain.
template <typename T>
__global__ void __launch_bounds__(kQuantThreads)
    fp8_quantize_tiles_kernel(const T *__restrict__ x, uint8_t *__restrict__ q, float *__restrict__ scale,
                              int64_t rows, int cols, int nb) {
    const int64_t br = blockIdx.x / nb;
    const int b = (int)(blockIdx.x - br * nb);
    const int64_t r0 = br * kF8Block;
    const int col = b * kF8Block + (threadIdx.x & 127);
    const int nr = (int)(rows - r0 < kF8Block ? rows - r0 : kF8Block);
    float top = 0.0f;
    if (col < cols)
        for (int r = threadIdx.x >> 7; r < nr; r += 2)
            top = fmaxf(top, finite_abs(to_f32(x[(r0 + r) * cols + col])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    __shared__ float tops[kQuantThreads / 32];
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQuantThreads / 32; ++i) top = fmaxf(top, tops[i]);
    const int p = f8_scale_exp(top);
    const float inv = pow2f(-p);
    if (col < cols)
        for (int r = threadIdx.x >> 7; r < nr; r += 2) {
            const int64_t at = (r0 + r) * cols + col;
            q[at] = (uint8_t)f8x2_satfinite(to_f32(x[at]) * inv, 0.0f);
        }
    if (threadIdx.x == 0) scale[blockIdx.x] = pow2f(p);
}

__global__ void __launch_bounds__(256)
    fp8_dequant_kernel(const uint8_t *__restrict__ q, const float *__restrict__ scale,
                       float *__restrict__ out, int64_t rows, int cols, int nb, int block_rows) {
    const int64_t n = rows * cols;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = i / cols;
        const int c = (int)(i - r * cols);
        const uint32_t h2 = [](uint32_t byte) {
            uint32_t r2;
            asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r2) : "r"(byte));
            return r2;
        }(q[i]);
        out[i] = half_bits_to_float(h2) * scale[(r / block_rows) * nb + c / kF8Block];
    }
}

template <typename T>
cudaError_t quantize(const T *x, uint8_t *q, float *scale, int64_t rows, int64_t cols, int block_rows,
                     cudaStream_t s) {
    const int64_t nb = f8_blocks(cols);
    if (block_rows != 1) {
        const int64_t tiles = f8_blocks(rows) * nb;
        if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
        fp8_quantize_tiles_kernel<T><<<(unsigned)tiles, kQuantThreads, 0, s>>>(x, q, scale, rows, (int)cols, (int)nb);
        return cudaGetLastError();
    }
    const int64_t units = rows * nb, per = kQuantThreads / 16;
    const int64_t grid = (units + per - 1) / per;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    const bool vec = ((reinterpret_cast<uintptr_t>(x) & 15) | (reinterpret_cast<uintptr_t>(q) & 7)) == 0 && cols % 8 == 0;
    if (vec)
        fp8_quantize_rows_kernel<T, true><<<(unsigned)grid, kQuantThreads, 0, s>>>(x, q, scale, rows, (int)cols, (int)nb);
    else
        fp8_quantize_rows_kernel<T, false><<<(unsigned)grid, kQuantThreads, 0, s>>>(x, q, scale, rows, (int)cols, (int)nb);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_quantize(int dtype, const void *x, uint8_t *q, float *scale, int64_t rows,
                                int64_t cols, int block_rows, cudaStream_t s) {
    if (dtype == ZFFN_DT_F32)
        return quantize(static_cast<const float *>(x), q, scale, rows, cols, block_rows, s);
    return quantize(static_cast<const __nv_bfloat16 *>(x), q, scale, rows, cols, block_rows, s);
}

cudaError_t launch_fp8_dequant(const uint8_t *q, const float *scale, float *out, int64_t rows,
                               int64_t cols, int block_rows, cudaStream_t s) {
    const int64_t n = rows * cols, blocks = (n + 255) / 256;
    fp8_dequant_kernel<<<(unsigned)(blocks < 65536 ? blocks : 65536), 256, 0, s>>>(
        q, scale, out, rows, (int)cols, (int)f8_blocks(cols), block_rows);
    return cudaGetLastError();
}

}  // namespace zffn
