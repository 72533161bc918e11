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

#include "launch.cuh"

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

// 1 x 128 blocks: 16 lanes per block, 8 columns per lane, UNITS blocks a thread
// with all of their loads in flight.  VEC: 16-byte loads and 8-byte stores (rows
// of 16-byte multiples from 16-byte aligned pointers); otherwise element by
// element.  WHOLE: the columns are a multiple of 128, so that blocks follow each
// other in memory (no division by the row's blocks).  Bound by HBM: 16384 x 2048 bf16
// takes 17.4 us, 5.8 TB/s.
template <typename T, bool VEC, bool WHOLE, int UNITS>
__global__ void __launch_bounds__(kQuantThreads)
    fp8_quantize_rows_kernel(const T *__restrict__ x, uint8_t *__restrict__ q, float *__restrict__ scale,
                             int64_t units, int cols, int nb) {
    grid_wait();
    grid_launch_dependents();
    constexpr int kPer = kQuantThreads / 16;
    const int sub = threadIdx.x & 15;
    const int64_t u0 = (int64_t)blockIdx.x * (kPer * UNITS) + (threadIdx.x >> 4);
    float v[UNITS][8];
    int64_t at[UNITS];    // element of the thread's first column
    int left[UNITS];      // columns of the row from there on
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
        const int64_t u = u0 + k * kPer;
        if (WHOLE) {
            at[k] = u * kF8Block + sub * 8;
            left[k] = u < units ? 8 : 0;
        } else {
            const int64_t row = u < 0x7fffffff ? (int64_t)((uint32_t)u / (uint32_t)nb) : u / nb;
            const int c0 = (int)(u - row * nb) * kF8Block + sub * 8;
            at[k] = row * cols + c0;
            left[k] = u < units ? cols - c0 : 0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = 0.0f;
        if (VEC) {
            if (left[k] > 0) load8(x + at[k], v[k]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left[k]) v[k][i] = to_f32(x[at[k] + i]);
        }
    }
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, finite_abs(v[k][i]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int p = f8_scale_exp(top);
        const float inv = pow2f(-p);
        const uint32_t lo = f8x4_satfinite(v[k][0] * inv, v[k][1] * inv, v[k][2] * inv, v[k][3] * inv);
        const uint32_t hi = f8x4_satfinite(v[k][4] * inv, v[k][5] * inv, v[k][6] * inv, v[k][7] * inv);
        if (VEC) {
            if (left[k] > 0) *reinterpret_cast<uint2 *>(q + at[k]) = make_uint2(lo, hi);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left[k]) q[at[k] + i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
        }
        const int64_t u = u0 + k * kPer;
        if (sub == 0 && u < units) scale[u] = pow2f(p);
    }
}

// 128 x 128 blocks: one thread block each; two passes over the block (the
// second from L1/L2), the maximum of the first between them.  Weights are
// quantised once, so this kernel is plain: 11008 x 4096 of fp32 takes 65 us, 3.5
// TB/s, of bf16 60 us, one element a load.
template <typename T>
__global__ void __launch_bounds__(kQuantThreads)
    fp8_quantize_tiles_kernel(const T *__restrict__ x, uint8_t *__restrict__ q, float *__restrict__ scale,
                              int64_t rows, int cols, int nb) {
    grid_wait();
    grid_launch_dependents();
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

// One element a thread and turn, two 64-bit divisions each: 11008 x 4096 takes 172
// us, 1.3 TB/s (no step of a layer dequantises).
__global__ void __launch_bounds__(256)
    fp8_dequant_kernel(const uint8_t *__restrict__ q, const float *__restrict__ scale,
                       float *__restrict__ out, int64_t rows, int cols, int nb, int block_rows) {
    grid_wait();
    grid_launch_dependents();
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
        return launch_dependent(fp8_quantize_tiles_kernel<T>, dim3((unsigned)tiles), kQuantThreads, 0, 1, s, x, q, scale, rows, cols, nb);
    }
    const int64_t units = rows * nb;
    const bool vec = ((reinterpret_cast<uintptr_t>(x) & 15) | (reinterpret_cast<uintptr_t>(q) & 7)) == 0 && cols % 8 == 0;
    // few blocks: one a thread, so that more SMs take part
    const bool few = units < (int64_t)(kQuantThreads / 16) * 4 * 1024;
    const int64_t per = kQuantThreads / 16 * (few ? 1 : 4), grid = (units + per - 1) / per;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    auto run = [&](auto kernel) { return launch_dependent(kernel, dim3((unsigned)grid), kQuantThreads, 0, 1, s, x, q, scale, units, cols, nb); };
    if (vec && cols % kF8Block == 0) return few ? run(fp8_quantize_rows_kernel<T, true, true, 1>) : run(fp8_quantize_rows_kernel<T, true, true, 4>);
    if (vec) return few ? run(fp8_quantize_rows_kernel<T, true, false, 1>) : run(fp8_quantize_rows_kernel<T, true, false, 4>);
    return few ? run(fp8_quantize_rows_kernel<T, false, false, 1>) : run(fp8_quantize_rows_kernel<T, false, false, 4>);
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
    return launch_dependent(fp8_dequant_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), 256, 0, 1, s, q, scale, out, rows, cols,
                            f8_blocks(cols), block_rows);
}

}  // namespace zffn
