// moe_sort.h -- launchers of moe_sort.cu: the sort of (token, slot) pairs by
// expert, rows to their sorted places and back, and the gradients.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace zffn {

cudaError_t launch_moe_sort(const int32_t *ids, int32_t *row_slot, int32_t *slot_row, int32_t *offsets,
                            int T, int E, int k, cudaStream_t s);
// a second array (scale, xs_scale: scale_bytes a row) moves with the first when scale_bytes > 0
cudaError_t launch_moe_dispatch(const void *x, int64_t row_bytes, const void *scale, int64_t scale_bytes,
                                const int32_t *row_slot, const int32_t *slot_row, void *xs, void *xs_scale,
                                int T, int k, cudaStream_t s);
// dtype: zffn_dtype of rows
cudaError_t launch_moe_combine(int dtype, const void *rows, const int32_t *slot_row, const float *weights,
                               float *y, int T, int H, int k, bool accumulate, cudaStream_t s);
cudaError_t launch_moe_combine_grad(int dtype, const float *dy, const void *rows, const int32_t *row_slot,
                                    const int32_t *slot_row, const float *weights, void *drows,
                                    float *dweights, int T, int H, int k, cudaStream_t s);

}  // namespace zffn
