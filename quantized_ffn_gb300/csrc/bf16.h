// bf16.h -- launchers of the bf16 products and their weights' gradients
// (bf16_matmul.cu), of SwiGLU (swiglu.cu) and of the low-rank adapters (lora.cu).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace zffn {

// y = a . w^T (w [E][N][K]) or a . w (transposed: w [E][K][N])
struct Bf16Args {
    const void *a;           // bf16 [M][K]
    const void *w;
    const int32_t *offsets;  // [E + 1] rows of each expert, or nullptr (dense)
    bool transposed;
    int y_dtype;             // zffn_dtype
    void *y;                 // [M][N]
    int M, N, K, E;
    int *err;
};
cudaError_t launch_bf16_matmul(const Bf16Args &a, cudaStream_t s);

// dw[e] = sum of dy[m]^T a[m] over expert e's rows
struct Bf16GradArgs {
    const void *dy;          // bf16 [M][N]
    const void *a;           // bf16 [M][K]
    const int32_t *offsets;
    int dw_dtype;
    void *dw;                // [E][N][K]
    int M, N, K, E;
    int *err;
};
cudaError_t launch_bf16_grad_w(const Bf16GradArgs &a, cudaStream_t s);

cudaError_t launch_swiglu(int dtype, const void *gu, void *h, int64_t rows, int64_t I, cudaStream_t s);
cudaError_t launch_swiglu_grad(int dtype, const void *dh, const void *gu, void *dgu, int64_t rows, int64_t I, cudaStream_t s);

// The tokens sorted by adapter.
struct LoraPlan {
    const int32_t *row_slot, *slot_row, *offsets;
    const float *scale;      // [L] or nullptr
    int T, r, L;
    int *err;
};
// Bytes of v's bf16 pieces, and whether a forward call goes row by row, without them.
size_t lora_pieces_bytes(int T, int r);
bool lora_by_rows(int T, int r, int L);
// v[row] = scale x[t] W^T, and its pieces v16: W [L][r][C], or (transposed) [L][C][r].  other:
// nullptr, or fp32 [T][r] whose pieces are written to other16 on the way.
cudaError_t launch_lora_shrink(const LoraPlan &p, const void *x, const void *w, bool transposed, float *v, void *v16, const float *other, void *other16,
                               int C, cudaStream_t s);
// out[t] = base[t] + v[row] W^T: W [L][C][r], or (transposed) [L][r][C].  Launched right after
// the shrink that writes v16.
cudaError_t launch_lora_expand(const LoraPlan &p, const void *v16, const void *w, bool transposed, int dtype, const void *base, void *out, int C,
                               cudaStream_t s);
// Both steps of the forward pass row by row.
cudaError_t launch_lora_rows(const LoraPlan &p, const void *x, const void *A, const void *B, int dtype, const void *base, void *out, float *v, int N, int K,
                             cudaStream_t s);
// dA[e] = sum of dv[row]^T x[t] over e's rows, [L][r][K], and dB[e] = sum of dy[t]^T v[row], [L][N][r]
cudaError_t launch_lora_outer(const LoraPlan &p, const void *dv16, const void *x, void *dA, int K, const void *v16, const void *dy, void *dB, int N, int dtype,
                              cudaStream_t s);

}  // namespace zffn
