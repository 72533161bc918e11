// swiglu.cu -- h = silu(g) u of rows [g | u], and its gradient.
#include "bf16.h"
#include "launch.cuh"

namespace zffn {
namespace {

template <typename T> __device__ __forceinline__ float load(const T *p);
template <> __device__ __forceinline__ float load(const float *p) { return *p; }
template <> __device__ __forceinline__ float load(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store(float *p, float v) { *p = v; }
__device__ __forceinline__ void store(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T>
__global__ void swiglu_kernel(const T *gu, T *h, int64_t rows, int64_t I) {
    const int64_t n = rows * I;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = i / I, c = i - r * I;
        const float g = load(gu + r * 2 * I + c), u = load(gu + r * 2 * I + I + c);
        store(h + i, g / (1.0f + expf(-g)) * u);
    }
}
template <typename T>
__global__ void swiglu_grad_kernel(const T *dh, const T *gu, T *dgu, int64_t rows, int64_t I) {
    const int64_t n = rows * I;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = i / I, c = i - r * I;
        const float g = load(gu + r * 2 * I + c), u = load(gu + r * 2 * I + I + c), d = load(dh + i);
        const float s = 1.0f / (1.0f + expf(-g));
        store(dgu + r * 2 * I + c, d * u * s * (1.0f + g * (1.0f - s)));
        store(dgu + r * 2 * I + I + c, d * g * s);
    }
}
unsigned grid_of(int64_t n) { return (unsigned)(n / 256 + 1 < 4096 ? n / 256 + 1 : 4096); }

}  // namespace

cudaError_t launch_swiglu(int dtype, const void *gu, void *h, int64_t rows, int64_t I, cudaStream_t s) {
    if (dtype == ZFFN_DT_BF16)
        swiglu_kernel<<<grid_of(rows * I), 256, 0, s>>>((const __nv_bfloat16 *)gu, (__nv_bfloat16 *)h, rows, I);
    else
        swiglu_kernel<<<grid_of(rows * I), 256, 0, s>>>((const float *)gu, (float *)h, rows, I);
    return cudaGetLastError();
}
cudaError_t launch_swiglu_grad(int dtype, const void *dh, const void *gu, void *dgu, int64_t rows, int64_t I, cudaStream_t s) {
    if (dtype == ZFFN_DT_BF16)
        swiglu_grad_kernel<<<grid_of(rows * I), 256, 0, s>>>((const __nv_bfloat16 *)dh, (const __nv_bfloat16 *)gu, (__nv_bfloat16 *)dgu, rows, I);
    else
        swiglu_grad_kernel<<<grid_of(rows * I), 256, 0, s>>>((const float *)dh, (const float *)gu, (float *)dgu, rows, I);
    return cudaGetLastError();
}

}  // namespace zffn
