// lora.cu -- low-rank adapters: products of rows grouped by adapter, and the sums of
// outer products over an adapter's rows.  One thread sums one value.
#include "bf16.h"
#include "launch.cuh"

namespace zffn {
namespace {

__device__ __forceinline__ float value(const void *p, int64_t i, bool bf16) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]) : static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void put(void *p, int64_t i, bool bf16, float v) {
    if (bf16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<float *>(p)[i] = v;
}
// First row of group g (g == E: of the rows of none): the largest offset up to it.
__device__ int first_row(const int32_t *offsets, int g, int E, int M) {
    if (!offsets) return g == 0 ? 0 : M;
    int lo = 0;
    for (int i = 0; i <= min(g, E); ++i) lo = max(lo, min(max(offsets[i], 0), M));
    return g > E ? M : lo;
}

struct Rows {
    const void *x, *w, *base;
    void *y;
    const int32_t *offsets, *in_row, *out_row, *slot_row;   // in_row, out_row: row -> row of x, of y (nullptr: itself)
    const float *scale;
    bool x_bf16, y_bf16;
    int M, N, K, E;
    int64_t wn, wk;   // strides of w by n and k
};
// y[out(m)][n] = base + scale sum_k x[in(m)][k] w[e][n][k]
__global__ void rows_kernel(const Rows p) {
    const int g = blockIdx.y, n = blockIdx.x * 32 + threadIdx.x;
    const int lo = first_row(p.offsets, g, p.E, p.M), hi = first_row(p.offsets, g + 1, p.E, p.M);
    if (n >= p.N) return;
    for (int m = lo + blockIdx.z * blockDim.y + threadIdx.y; m < hi; m += gridDim.z * blockDim.y) {
        const int in = p.in_row ? p.in_row[m] : m, out = p.out_row ? p.out_row[m] : m;
        const bool some = g < p.E && (unsigned)in < (unsigned)p.M;
        float sum = 0.0f;
        if (some)
            for (int k = 0; k < p.K; ++k)
                sum += value(p.x, (int64_t)in * p.K + k, p.x_bf16) * value(p.w, (int64_t)g * p.N * p.K + n * p.wn + k * p.wk, true);
        if (p.scale && some) sum *= p.scale[g];
        if ((unsigned)out >= (unsigned)p.M || (p.out_row && !some)) continue;
        const int64_t at = (int64_t)out * p.N + n;
        put(p.y, at, p.y_bf16, (p.base ? value(p.base, at, p.y_bf16) : 0.0f) + sum);
    }
}
// tokens of no adapter: y = base or 0
__global__ void rest_kernel(const Rows p) {
    const int n = blockIdx.x * 32 + threadIdx.x;
    if (n >= p.N) return;
    for (int t = blockIdx.z * blockDim.y + threadIdx.y; t < p.M; t += gridDim.z * blockDim.y)
        if (p.slot_row[t] < 0) put(p.y, (int64_t)t * p.N + n, p.y_bf16, p.base ? value(p.base, (int64_t)t * p.N + n, p.y_bf16) : 0.0f);
}
cudaError_t launch_rows(const Rows &p, cudaStream_t s) {
    const dim3 grid((p.N + 31) / 32, p.E + (p.offsets ? 1 : 0), p.M / p.E / 8 + 1 < 64 ? p.M / p.E / 8 + 1 : 64);
    rows_kernel<<<grid, dim3(32, 8), 0, s>>>(p);
    if (p.slot_row && p.y != p.base) rest_kernel<<<dim3((p.N + 31) / 32, 1, 64), dim3(32, 8), 0, s>>>(p);
    return cudaGetLastError();
}

struct Outer {
    const void *a, *b;
    void *d;
    const int32_t *offsets, *a_row, *b_row;
    bool a_bf16, b_bf16, d_bf16;
    int M, NA, NB, E;
};
// d[e][i][j] = sum over e's rows of a[.][i] b[.][j]
__global__ void outer_kernel(const Outer p) {
    const int g = blockIdx.z;
    const int lo = first_row(p.offsets, g, p.E, p.M), hi = first_row(p.offsets, g + 1, p.E, p.M);
    const int j = blockIdx.x * 32 + threadIdx.x;
    for (int i = blockIdx.y * 8 + threadIdx.y; i < p.NA; i += gridDim.y * 8) {
        if (j >= p.NB) return;
        float sum = 0.0f;
        for (int m = lo; m < hi; ++m) {
            const int ra = p.a_row ? p.a_row[m] : m, rb = p.b_row ? p.b_row[m] : m;
            if ((unsigned)ra >= (unsigned)p.M || (unsigned)rb >= (unsigned)p.M) continue;
            sum += value(p.a, (int64_t)ra * p.NA + i, p.a_bf16) * value(p.b, (int64_t)rb * p.NB + j, p.b_bf16);
        }
        put(p.d, ((int64_t)g * p.NA + i) * p.NB + j, p.d_bf16, sum);
    }
}
cudaError_t launch_outer(const Outer &p, cudaStream_t s) {
    outer_kernel<<<dim3((p.NB + 31) / 32, (p.NA + 7) / 8, p.E), dim3(32, 8), 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lora_shrink(const LoraPlan &p, const void *x, const void *w, bool transposed, float *v, int C, cudaStream_t s) {
    return launch_rows({x, w, nullptr, v, p.offsets, p.row_slot, nullptr, nullptr, p.scale, true, false, p.T, p.r, C, p.L,
                        transposed ? 1 : C, transposed ? p.r : 1}, s);
}
cudaError_t launch_lora_expand(const LoraPlan &p, const float *v, const void *w, bool transposed, int dtype, const void *base, void *out,
                               int C, cudaStream_t s) {
    return launch_rows({v, w, base, out, p.offsets, nullptr, p.row_slot, p.slot_row, nullptr, false, dtype == ZFFN_DT_BF16, p.T, C, p.r, p.L,
                        transposed ? 1 : p.r, transposed ? C : 1}, s);
}
cudaError_t launch_lora_outer(const LoraPlan &p, const float *v, const void *x, bool transposed, int dtype, void *d, int C, cudaStream_t s) {
    if (transposed) return launch_outer({x, v, d, p.offsets, p.row_slot, nullptr, true, false, dtype == ZFFN_DT_BF16, p.T, C, p.r, p.L}, s);
    return launch_outer({v, x, d, p.offsets, nullptr, p.row_slot, false, true, dtype == ZFFN_DT_BF16, p.T, p.r, C, p.L}, s);
}

}  // namespace zffn
