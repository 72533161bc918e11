// api_bf16.cu -- C ABI of the bf16 products, SwiGLU and low-rank adapters: host-side
// argument checks and the composition of the launches.
#include "bf16.h"
#include "launch.cuh"

namespace zffn {
namespace {

inline uintptr_t bits(const void *p) { return reinterpret_cast<uintptr_t>(p); }
inline size_t dtype_bytes(int dtype) { return dtype == ZFFN_DT_BF16 ? 2 : 4; }
inline bool dtype_valid(int dtype) { return dtype == ZFFN_DT_F32 || dtype == ZFFN_DT_BF16; }

zffn_status check_product(const int32_t *offsets, int M, int N, int K, int E, bool n8) {
    if (M < 1 || M > (1 << 24) || N < 1 || N > 65536) return invalid("M must be in [1, 2^24] and N in [1, 65536]");
    if (K < 8 || K > 65536 || K % 8) return invalid("K must be a multiple of 8 in [8, 65536]");
    if (n8 && N % 8) return invalid("N must be a multiple of 8");
    if (E < 1 || E > 4096 || (!offsets && E != 1)) return invalid("E must be in [1, 4096], and 1 without offsets");
    if (bits(offsets) & 3) return invalid("offsets must be 4-byte aligned");
    return ZFFN_OK;
}

zffn_status check_swiglu(int dtype, const void *a, const void *b, const void *c, int64_t rows, int64_t I) {
    if (!dtype_valid(dtype)) return invalid("unknown dtype");
    if (!a || !b || !c) return invalid("a pointer argument is NULL");
    if (rows < 1 || rows > 0x7fffffff || I < 1 || I > (1 << 20)) return invalid("rows must be in [1, 2^31 - 1] and I in [1, 2^20]");
    if ((bits(a) | bits(b) | bits(c)) & (dtype_bytes(dtype) - 1)) return invalid("the pointers must be aligned to their element");
    return ZFFN_OK;
}

zffn_status check_lora(const LoraPlan &p, int N, int K) {
    if (!p.row_slot || !p.slot_row || !p.offsets) return invalid("a pointer argument is NULL");
    if (p.T < 1 || p.T > (1 << 24)) return invalid("T must be in [1, 2^24]");
    if (N < 8 || N > 65536 || N % 8 || K < 8 || K > 65536 || K % 8) return invalid("N and K must be multiples of 8 in [8, 65536]");
    if (p.r < 8 || p.r > 128 || p.r % 8) return invalid("r must be a multiple of 8 in [8, 128]");
    if (p.L < 1 || p.L > 4096) return invalid("L must be in [1, 4096]");
    if ((bits(p.row_slot) | bits(p.slot_row) | bits(p.offsets) | bits(p.scale)) & 3)
        return invalid("row_slot, slot_row, offsets and scale must be 4-byte aligned");
    return ZFFN_OK;
}

}  // namespace
}  // namespace zffn

using namespace zffn;

extern "C" {

zffn_status zffn_bf16_matmul(const void *a, const void *w, const int32_t *offsets, int transposed, int y_dtype, void *y,
                             int M, int N, int K, int E, void *stream) {
    if (!a || !w || !y) return invalid("a pointer argument is NULL");
    if (!dtype_valid(y_dtype)) return invalid("unknown y_dtype");
    if (check_product(offsets, M, N, K, E, transposed != 0) != ZFFN_OK) return ZFFN_ERR_INVALID_ARG;
    if ((bits(a) | bits(w)) & 15) return invalid("a and w must be 16-byte aligned");
    if (bits(y) & (dtype_bytes(y_dtype) - 1)) return invalid("y must be aligned to its element");
    const DeviceInfo &di = device_info();
    if (di.device < 0) return ZFFN_ERR_CUDA;
    return to_status(launch_bf16_matmul({a, w, offsets, transposed != 0, y_dtype, y, M, N, K, E, di.err_word}, (cudaStream_t)stream));
}

zffn_status zffn_bf16_matmul_grad_w(const void *dy, const void *a, const int32_t *offsets, int dw_dtype, void *dw, int M,
                                    int N, int K, int E, void *stream) {
    if (!dy || !a || !dw) return invalid("a pointer argument is NULL");
    if (!dtype_valid(dw_dtype)) return invalid("unknown dw_dtype");
    if (check_product(offsets, M, N, K, E, true) != ZFFN_OK) return ZFFN_ERR_INVALID_ARG;
    if ((bits(dy) | bits(a) | bits(dw)) & 15) return invalid("dy, a and dw must be 16-byte aligned");
    const DeviceInfo &di = device_info();
    if (di.device < 0) return ZFFN_ERR_CUDA;
    return to_status(launch_bf16_grad_w({dy, a, offsets, dw_dtype, dw, M, N, K, E, di.err_word}, (cudaStream_t)stream));
}

zffn_status zffn_swiglu(int dtype, const void *gu, void *h, int64_t rows, int64_t I, void *stream) {
    if (check_swiglu(dtype, gu, h, h, rows, I) != ZFFN_OK) return ZFFN_ERR_INVALID_ARG;
    if (device_info().device < 0) return ZFFN_ERR_CUDA;
    return to_status(launch_swiglu(dtype, gu, h, rows, I, (cudaStream_t)stream));
}

zffn_status zffn_swiglu_grad(int dtype, const void *dh, const void *gu, void *dgu, int64_t rows, int64_t I, void *stream) {
    if (check_swiglu(dtype, dh, gu, dgu, rows, I) != ZFFN_OK) return ZFFN_ERR_INVALID_ARG;
    if (device_info().device < 0) return ZFFN_ERR_CUDA;
    return to_status(launch_swiglu_grad(dtype, dh, gu, dgu, rows, I, (cudaStream_t)stream));
}

size_t zffn_lora_work_bytes(int T, int r, int L, int backward) {
    if (T < 1 || T > (1 << 24) || r < 8 || r > 128 || r % 8 || L < 1 || L > 4096) return 0;
    return backward ? 2 * lora_pieces_bytes(T, r) : lora_by_rows(T, r, L) ? 0 : lora_pieces_bytes(T, r);
}

zffn_status zffn_lora_add(const void *x, const void *A, const void *B, const float *scale, const int32_t *row_slot,
                          const int32_t *slot_row, const int32_t *offsets, int dtype, const void *base, void *out, float *v,
                          void *work, int T, int N, int K, int r, int L, void *stream) {
    LoraPlan p{row_slot, slot_row, offsets, scale, T, r, L, nullptr};
    if (!x || !A || !B || !out || !v) return invalid("a pointer argument is NULL");
    if (!dtype_valid(dtype)) return invalid("unknown dtype");
    if (check_lora(p, N, K) != ZFFN_OK) return ZFFN_ERR_INVALID_ARG;
    const bool by_rows = lora_by_rows(T, r, L);
    if (!work && !by_rows) return invalid("work is NULL");
    if ((bits(x) | bits(A) | bits(B) | bits(base) | bits(out) | bits(v) | bits(work)) & 15)
        return invalid("x, A, B, base, out, v and work must be 16-byte aligned");
    const DeviceInfo &di = device_info();
    if (di.device < 0) return ZFFN_ERR_CUDA;
    p.err = di.err_word;
    cudaStream_t s = (cudaStream_t)stream;
    if (by_rows) return to_status(launch_lora_rows(p, x, A, B, dtype, base, out, v, N, K, s));
    const cudaError_t e = launch_lora_shrink(p, x, A, false, v, work, nullptr, nullptr, K, s);
    if (e != cudaSuccess) return to_status(e);
    return to_status(launch_lora_expand(p, work, B, false, dtype, base, out, N, s));
}

zffn_status zffn_lora_grad(const void *dy, const void *x, const float *v, const void *A, const void *B, const float *scale,
                           const int32_t *row_slot, const int32_t *slot_row, const int32_t *offsets, int dx_dtype,
                           const void *base, void *dx, int dw_dtype, void *dA, void *dB, float *dv, void *work, int T,
                           int N, int K, int r, int L, void *stream) {
    LoraPlan p{row_slot, slot_row, offsets, scale, T, r, L, nullptr};
    if (!dy || !x || !v || !A || !B || !dx || !dA || !dB || !dv || !work) return invalid("a pointer argument is NULL");
    if (!dtype_valid(dx_dtype) || !dtype_valid(dw_dtype)) return invalid("unknown dtype");
    if (check_lora(p, N, K) != ZFFN_OK) return ZFFN_ERR_INVALID_ARG;
    if ((bits(dy) | bits(x) | bits(v) | bits(A) | bits(B) | bits(base) | bits(dx) | bits(dA) | bits(dB) | bits(dv) | bits(work)) & 15)
        return invalid("dy, x, v, A, B, base, dx, dA, dB, dv and work must be 16-byte aligned");
    const DeviceInfo &di = device_info();
    if (di.device < 0) return ZFFN_ERR_CUDA;
    p.err = di.err_word;
    cudaStream_t s = (cudaStream_t)stream;
    uint8_t *dv16 = static_cast<uint8_t *>(work), *v16 = dv16 + lora_pieces_bytes(T, r);
    cudaError_t e = launch_lora_shrink(p, dy, B, true, dv, dv16, v, v16, N, s);
    if (e == cudaSuccess) e = launch_lora_expand(p, dv16, A, true, dx_dtype, base, dx, K, s);
    if (e == cudaSuccess) e = launch_lora_outer(p, dv16, x, dA, K, v16, dy, dB, N, dw_dtype, s);
    return to_status(e);
}

}  // extern "C"
