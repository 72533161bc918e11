// swiglu.cu -- h = silu(g) u of rows [g | u], and its gradient.  One pass: each value is
// read once and written once, a thread's two or four accesses of each kind before the
// first sum.  Bound by HBM: 32768 rows of 768 bf16 (151 MB) take 22.9 us, 6.6 TB/s, their
// gradient (252 MB) 37.1 us, 6.8 TB/s.
#include "bf16.h"
#include "groups.cuh"
#include "launch.cuh"

namespace zffn {
namespace {

constexpr int THREADS = 256;
// Packs a thread has on their way: two of 16 bytes (four: 29.2 and 52.0 us for the rows above,
// fewer threads an SM; one 22.6 and 37.2), four of narrower ones (1859 x 1021 of fp32, forward:
// 4.6 us, two 5.0, one 8.6).
constexpr int together(int bytes) { return bytes == 16 ? 2 : 4; }

// 1 / (1 + e^-g).  fp32: by the exponential and the division of the language.  bf16: by the
// special function unit's two instructions (off by (3 + |g| / 3) 2^-22 of the value at most,
// and 0 below g = -87.3, where silu is above -1.1e-36), since a result keeps 2^-8: the other
// form's 40 instructions a value would take longer than its bytes (27 us for 32768 x 768).
template <typename T> __device__ __forceinline__ float logistic(float g);
template <> __device__ __forceinline__ float logistic<float>(float g) { return 1.0f / (1.0f + expf(-g)); }
template <> __device__ __forceinline__ float logistic<__nv_bfloat16>(float g) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// V values at once
template <typename T, int V> struct alignas(sizeof(T) * V) Pack { T v[V]; };
__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float &to, float x) { to = x; }
__device__ __forceinline__ void put(__nv_bfloat16 &to, float x) { to = __float2bfloat16_rn(x); }

// `cols`: packs of a row of I values; n: packs of all rows
template <typename T, int V>
__global__ void __launch_bounds__(THREADS) swiglu_kernel(const Pack<T, V> *gu, Pack<T, V> *h, FastDiv cols, int n) {
    constexpr int TOGETHER = together(sizeof(T) * V);
    grid_wait();
    grid_launch_dependents();
    const int first = blockIdx.x * (THREADS * TOGETHER) + threadIdx.x;
    Pack<T, V> g[TOGETHER], u[TOGETHER];
#pragma unroll
    for (int k = 0; k < TOGETHER; ++k) {
        const int i = first + k * THREADS;
        if (i >= n) break;
        const int64_t at = i + (int64_t)cols.div(i) * cols.d;    // (a row of gu has 2 I values)
        g[k] = gu[at];
        u[k] = gu[at + cols.d];
    }
#pragma unroll
    for (int k = 0; k < TOGETHER; ++k) {
        const int i = first + k * THREADS;
        if (i >= n) break;
        Pack<T, V> out;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float x = value(g[k].v[j]);
            put(out.v[j], x * logistic<T>(x) * value(u[k].v[j]));
        }
        h[i] = out;
    }
}

// (dgu may be gu: a thread writes only what it alone has read)
template <typename T, int V>
__global__ void __launch_bounds__(THREADS) swiglu_grad_kernel(const Pack<T, V> *dh, const Pack<T, V> *gu, Pack<T, V> *dgu, FastDiv cols, int n) {
    constexpr int TOGETHER = together(sizeof(T) * V);
    grid_wait();
    grid_launch_dependents();
    const int first = blockIdx.x * (THREADS * TOGETHER) + threadIdx.x;
    Pack<T, V> g[TOGETHER], u[TOGETHER], d[TOGETHER];
    int64_t at[TOGETHER];
#pragma unroll
    for (int k = 0; k < TOGETHER; ++k) {
        const int i = first + k * THREADS;
        if (i >= n) break;
        at[k] = i + (int64_t)cols.div(i) * cols.d;
        g[k] = gu[at[k]];
        u[k] = gu[at[k] + cols.d];
        d[k] = dh[i];
    }
#pragma unroll
    for (int k = 0; k < TOGETHER; ++k) {
        const int i = first + k * THREADS;
        if (i >= n) break;
        Pack<T, V> dg, du;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float x = value(g[k].v[j]), s = logistic<T>(x), y = value(d[k].v[j]);
            // (the slope first, at most 1.1: a product of dh and u or g could overflow where the result does not)
            put(dg.v[j], y * (value(u[k].v[j]) * (s * (1.0f + x * (1.0f - s)))));
            put(du.v[j], y * (x * s));
        }
        dgu[at[k]] = dg;
        dgu[at[k] + cols.d] = du;
    }
}

// Packs of V values where I and every pointer allow them; at most 2^30 packs a launch.
template <typename T, int V>
cudaError_t run(const void *dh, const void *gu, void *out, int64_t rows, int64_t I, cudaStream_t s) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(dh) | reinterpret_cast<uintptr_t>(gu) | reinterpret_cast<uintptr_t>(out);
    if constexpr (V > 1) {
        if (I % V || (bits & (sizeof(T) * V - 1))) return run<T, V / 2>(dh, gu, out, rows, I, s);
    }
    using P = Pack<T, V>;
    constexpr int TOGETHER = together(sizeof(T) * V);
    const int64_t cols = I / V, most = (1 << 30) / cols;
    for (int64_t r = 0; r < rows; r += most) {
        const int64_t n = (rows - r < most ? rows - r : most) * cols;
        const dim3 grid((unsigned)((n + THREADS * TOGETHER - 1) / (THREADS * TOGETHER)));
        const P *from = static_cast<const P *>(gu) + r * 2 * cols;
        cudaError_t e;
        if (dh)
            e = launch_dependent(swiglu_grad_kernel<T, V>, grid, THREADS, 0, 1, s, static_cast<const P *>(dh) + r * cols, from,
                                 static_cast<P *>(out) + r * 2 * cols, FastDiv((uint32_t)cols), (int)n);
        else
            e = launch_dependent(swiglu_kernel<T, V>, grid, THREADS, 0, 1, s, from, static_cast<P *>(out) + r * cols, FastDiv((uint32_t)cols), (int)n);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_swiglu(int dtype, const void *gu, void *h, int64_t rows, int64_t I, cudaStream_t s) {
    return dtype == ZFFN_DT_BF16 ? run<__nv_bfloat16, 8>(nullptr, gu, h, rows, I, s) : run<float, 4>(nullptr, gu, h, rows, I, s);
}
cudaError_t launch_swiglu_grad(int dtype, const void *dh, const void *gu, void *dgu, int64_t rows, int64_t I, cudaStream_t s) {
    return dtype == ZFFN_DT_BF16 ? run<__nv_bfloat16, 8>(dh, gu, dgu, rows, I, s) : run<float, 4>(dh, gu, dgu, rows, I, s);
}

}  // namespace zffn
