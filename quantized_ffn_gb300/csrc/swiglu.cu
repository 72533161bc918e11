// swiglu.cu -- h = silu(g) u of rows [g | u], and its gradient.  One pass: each value is
// read once and written once, a thread's two or four accesses of each kind before the
// first sum.  Bound by HBM: 32768 rows of 768 bf16 (151 MB) take 22.4 us, 6.7 TB/s, their
// gradient (252 MB) 37.3 us, 6.8 TB/s.
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

// 1 / (1 + e^-g) for g >= FAR.  fp32: by the exponential and the division of the language.  bf16:
// by the special function unit's two instructions (off by (3 + |g| / 3) 2^-22 of the value at
// most), since a result keeps 2^-8: the other form's 40 instructions a value would take longer
// than its bytes (27 us for 32768 x 768).
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

// Below FAR (which a gate seldom reaches) 1 / (1 + e^-g) is e^g to 2^-46 of it, and may be far below
// fp32's range where its product with a large u or dh is within it: a pack that holds such a g
// goes value by value, with products in 64 bits for those.  (A quarter's exponential is a
// normal number down to g = -349, where no product of two fp32 values brings it back.)  The
// values are read again: kept in registers they took 8 to 12 of the others' room.  Asking costs
// rows of whole packs nothing (32768 x 768 bf16: 22.1 / 22.4 us), odd ones some 5 % (1859 x 1021 fp32:
// 4.6 / 4.8 us, the gradient 5.8 / 6.0; 32768 x 767 bf16 31.8 / 34.3); with a far gate in a thousand
// 32768 x 768 bf16 take 28 us.
constexpr float FAR = -32.0f;
__device__ __forceinline__ double far_logistic(float g) {
    const double q = expf(0.25f * g);
    return (q * q) * (q * q);
}
template <typename T, int V> __device__ __forceinline__ bool any_far(const Pack<T, V> &g) {
    float least = value(g.v[0]);
#pragma unroll
    for (int j = 1; j < V; ++j) least = fminf(least, value(g.v[j]));
    return least < FAR;
}
template <typename T> __device__ __forceinline__ float forward(float x, float u) { return x * logistic<T>(x) * u; }
// The slope first, at most 1.1: a product of dh and u or g could overflow where the result does not.
template <typename T> __device__ __forceinline__ float2 backward(float x, float u, float y) {
    const float s = logistic<T>(x);
    return make_float2(y * (u * (s * (1.0f + x * (1.0f - s)))), y * (x * s));
}
template <typename T, int V> __device__ __forceinline__ void far_forward(const T *g, const T *u, T *h) {
#pragma unroll 1
    for (int j = 0; j < V; ++j) {
        const float x = value(g[j]), v = value(u[j]);
        put(h[j], x < FAR ? (float)(x * far_logistic(x) * v) : forward<T>(x, v));
    }
}
template <typename T, int V> __device__ __forceinline__ void far_backward(const T *dh, const T *g, const T *u, T *dg, T *du) {
#pragma unroll 1
    for (int j = 0; j < V; ++j) {
        const float x = value(g[j]), v = value(u[j]), y = value(dh[j]);
        float2 d;
        if (x < FAR) {
            const double ys = y * far_logistic(x);
            d = make_float2((float)(ys * v * (1.0 + x)), (float)(ys * x));
        } else {
            d = backward<T>(x, v, y);
        }
        put(dg[j], d.x);
        put(du[j], d.y);
    }
}

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
        if (any_far(g[k])) {
            const Pack<T, V> *from = gu + i + (int64_t)cols.div(i) * cols.d;
            far_forward<T, V>(from->v, from[cols.d].v, h[i].v);
            continue;
        }
        Pack<T, V> out;
#pragma unroll
        for (int j = 0; j < V; ++j) put(out.v[j], forward<T>(value(g[k].v[j]), value(u[k].v[j])));
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
        if (any_far(g[k])) {
            far_backward<T, V>(dh[i].v, gu[at[k]].v, gu[at[k] + cols.d].v, dgu[at[k]].v, dgu[at[k] + cols.d].v);
            continue;
        }
        Pack<T, V> dg, du;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 both = backward<T>(value(g[k].v[j]), value(u[k].v[j]), value(d[k].v[j]));
            put(dg.v[j], both.x);
            put(du.v[j], both.y);
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
