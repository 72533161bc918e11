// fp8_matmul.cu -- products of block-scaled e4m3 matrices, dense or grouped by
// expert, plain or with SwiGLU and quantisation of the result.
//
// One warp per output block of 1 row x 128 columns; every lane sums four
// columns over K on the CUDA cores.  The simplest form that covers every size.
#include "fp8.h"
#include "zffn_internal.cuh"

namespace zffn {

namespace {

__device__ __forceinline__ void f8x4_to_f32(uint32_t v, float (&f)[4]) {
    uint32_t a, b;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(v));
    f[0] = half_bits_to_float(a); f[1] = half_bits_to_float(a >> 16);
    f[2] = half_bits_to_float(b); f[3] = half_bits_to_float(b >> 16);
}

// sum over K of row m of a and row n of expert e's w, with both scales
__device__ float dot_row(const uint8_t *a, const float *as, const uint8_t *w, const float *ws, int K) {
    float acc = 0.0f;
    for (int b = 0; b * kF8Block < K; ++b) {
        const int k1 = min(K, (b + 1) * kF8Block);
        float s = 0.0f;
        for (int k = b * kF8Block; k < k1; k += 4) {
            float x[4], y[4];
            f8x4_to_f32(*reinterpret_cast<const uint32_t *>(a + k), x);
            f8x4_to_f32(*reinterpret_cast<const uint32_t *>(w + k), y);
#pragma unroll
            for (int i = 0; i < 4; ++i) s = fmaf(x[i], y[i], s);
        }
        acc = fmaf(s, as[b] * ws[b], acc);
    }
    return acc;
}

__global__ void __launch_bounds__(128) fp8_matmul_kernel(Fp8Args p) {
    const int nb = (int)f8_blocks(p.N), kb = (int)f8_blocks(p.K), lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t m = unit / nb;
    const int b = (int)(unit - m * nb);
    if (m >= p.M) return;
    int e = 0;
    if (p.offsets) {
        while (e < p.E && !(m >= p.offsets[e] && m < p.offsets[e + 1])) ++e;
    }
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = 0; i < 4 && e < p.E; ++i) {
        const int n = b * kF8Block + lane * 4 + i;
        if (n >= p.N) continue;
        const int64_t row = (int64_t)e * p.N + n, srow = ((int64_t)e * nb + b) * kb;
        v[i] = dot_row(p.a + m * p.K, p.a_scale + m * kb, p.w + row * p.K, p.w_scale + srow, p.K);
        if (p.w1) {
            const float u = dot_row(p.a + m * p.K, p.a_scale + m * kb, p.w1 + row * p.K, p.w1_scale + srow, p.K);
            v[i] = __fdividef(v[i], 1.0f + __expf(-v[i])) * u;
        }
    }
    int sp = 0;
    if (p.w1) {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, finite_abs(v[i]));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        sp = f8_scale_exp(top);
        if (lane == 0) p.y_scale[m * nb + b] = pow2f(sp);
    }
    for (int i = 0; i < 4; ++i) {
        const int n = b * kF8Block + lane * 4 + i;
        if (n >= p.N) continue;
        const int64_t at = m * p.N + n;
        if (p.w1) static_cast<uint8_t *>(p.y)[at] = (uint8_t)f8x2_satfinite(v[i] * pow2f(-sp), 0.0f);
        else if (p.y_dtype == ZFFN_DT_F32) static_cast<float *>(p.y)[at] = v[i];
        else static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(v[i]);
    }
}

}  // namespace

cudaError_t launch_fp8_matmul(const Fp8Args &a, cudaStream_t s) {
    const int64_t units = (int64_t)a.M * f8_blocks(a.N), grid = (units + 3) / 4;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    fp8_matmul_kernel<<<(unsigned)grid, 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace zffn
