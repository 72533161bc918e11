// api_fp8.cu -- C ABI of the block-scaled 8-bit entry points and of the sort by
// expert: host-side argument checks and the composition of the launches.
#include "fp8.h"
#include "moe_sort.h"
#include "launch.cuh"

namespace zffn {

namespace {

inline uintptr_t bits(const void *p) { return reinterpret_cast<uintptr_t>(p); }
inline size_t align_up(size_t v) { return (v + 255) / 256 * 256; }
inline size_t dtype_bytes(int dtype) { return dtype == ZFFN_DT_BF16 ? 2 : 4; }
inline bool dtype_valid(int dtype) { return dtype == ZFFN_DT_F32 || dtype == ZFFN_DT_BF16; }

// Sub-buffers of the workspace: h of the experts' products, and what the routed
// block keeps between its steps.  The first 256 bytes are the one-launch routed
// path's.
struct F8Layout {
    size_t h, hs, q, qs, xq, xs, rows, row_slot, slot_row, offsets, total;
};
F8Layout f8_layout(int64_t P, int T, int H, int I, int E) {
    F8Layout L;
    size_t o = 256;
    L.h = o; o = align_up(o + (size_t)P * I);
    L.hs = o; o = align_up(o + (size_t)P * f8_blocks(I) * 4);
    L.q = o; o = align_up(o + (size_t)T * H);
    L.qs = o; o = align_up(o + (size_t)T * f8_blocks(H) * 4);
    L.xq = o; o = align_up(o + (size_t)P * H);
    L.xs = o; o = align_up(o + (size_t)P * f8_blocks(H) * 4);
    L.rows = o; o = align_up(o + (size_t)P * H * 2);
    L.row_slot = o; o = align_up(o + (size_t)P * 4);
    L.slot_row = o; o = align_up(o + (size_t)P * 4);
    L.offsets = o; o = align_up(o + (size_t)(E + 1) * 4);
    L.total = o;
    return L;
}
size_t experts_bytes(int64_t P, int I) { return align_up(align_up(256 + (size_t)P * I) + (size_t)P * f8_blocks(I) * 4); }

zffn_status check_quant(const void *q, const float *scale, const void *x, size_t x_size, int64_t rows, int64_t cols,
                        int block_rows) {
    if (!q || !scale || !x) return invalid("a pointer argument is NULL");
    if (rows < 1 || rows > 0x7fffffff || cols < 1 || cols > (1 << 20))
        return invalid("rows must be in [1, 2^31 - 1] and cols in [1, 2^20]");
    if (block_rows != 1 && block_rows != 128) return invalid("block_rows must be 1 or 128");
    if ((bits(x) & (x_size - 1)) || (bits(scale) & 3)) return invalid("x must be aligned to its element and scale to 4 bytes");
    return ZFFN_OK;
}

zffn_status check_route(int T, int E, int k) {
    if (T < 1 || E < 1 || E > 4096 || k < 1 || k > 64) return invalid("T >= 1, E in [1, 4096] and top_k in [1, 64] are required");
    if ((int64_t)T * k > (1 << 24)) return invalid("T * top_k must not exceed 2^24");
    return ZFFN_OK;
}

// h (in the workspace at h, hs) and y of the experts' two products
zffn_status run_experts(const uint8_t *a, const float *a_scale, const int32_t *offsets, const void *Wg, const float *sg,
                        const void *Wu, const float *su, const void *Wd, const float *sd, int y_dtype, void *y, int P,
                        int H, int I, int E, uint8_t *h, float *hs, int *err, cudaStream_t s) {
    Fp8Args g{};
    g.a = a;
    g.a_scale = a_scale;
    g.offsets = offsets;
    g.w = static_cast<const uint8_t *>(Wg);
    g.w_scale = sg;
    g.w1 = static_cast<const uint8_t *>(Wu);
    g.w1_scale = su;
    g.y = h;
    g.y_scale = hs;
    g.M = P; g.N = I; g.K = H; g.E = E;
    g.err = err;
    const cudaError_t e = launch_fp8_matmul(g, s);
    if (e != cudaSuccess) return to_status(e);
    Fp8Args d{};
    d.a = h;
    d.a_scale = hs;
    d.offsets = offsets;
    d.w = static_cast<const uint8_t *>(Wd);
    d.w_scale = sd;
    d.y = y;
    d.y_dtype = y_dtype;
    d.M = P; d.N = H; d.K = I; d.E = E;
    d.err = err;
    d.early = true;   // (the product before writes h and its scales)
    return to_status(launch_fp8_matmul(d, s));
}

zffn_status check_experts(int64_t P, int H, int I, int E) {
    if (P < 1 || P > (1 << 24)) return invalid("the number of rows must be in [1, 2^24]");
    if (H < 16 || H > 65536 || H % 16 || I < 16 || I > 65536 || I % 16)
        return invalid("H and I must be multiples of 16 in [16, 65536]");
    if (E < 1 || E > 4096) return invalid("E must be in [1, 4096]");
    if ((int64_t)E * (H > I ? H : I) > 0x7fffffff) return invalid("E * max(H, I) must be below 2^31");
    return ZFFN_OK;
}

}  // namespace

size_t fp8_workspace_bytes(int T, int H, int I, int E, int k) {
    return f8_layout((int64_t)T * k, T, H, I, E).total;
}

}  // namespace zffn

using namespace zffn;

extern "C" {

zffn_status zffn_fp8_quantize(int dtype, const void *x, void *q, float *scale, int64_t rows, int64_t cols,
                              int block_rows, void *stream) {
    if (!dtype_valid(dtype)) return invalid("unknown dtype");
    const zffn_status st = check_quant(q, scale, x, dtype_bytes(dtype), rows, cols, block_rows);
    if (st != ZFFN_OK) return st;
    if (device_info().device < 0) return ZFFN_ERR_CUDA;
    return to_status(launch_fp8_quantize(dtype, x, static_cast<uint8_t *>(q), scale, rows, cols, block_rows, (cudaStream_t)stream));
}

zffn_status zffn_fp8_dequant(const void *q, const float *scale, float *out, int64_t rows, int64_t cols, int block_rows,
                             void *stream) {
    const zffn_status st = check_quant(q, scale, out, 4, rows, cols, block_rows);
    if (st != ZFFN_OK) return st;
    if (device_info().device < 0) return ZFFN_ERR_CUDA;
    return to_status(launch_fp8_dequant(static_cast<const uint8_t *>(q), scale, out, rows, cols, block_rows, (cudaStream_t)stream));
}

zffn_status zffn_fp8_matmul(const void *a, const float *a_scale, const void *w, const float *w_scale,
                            const int32_t *offsets, int y_dtype, void *y, int M, int N, int K, int E, void *stream) {
    if (!a || !a_scale || !w || !w_scale || !y) return invalid("a pointer argument is NULL");
    if (!dtype_valid(y_dtype)) return invalid("unknown y_dtype");
    if (M < 1 || M > (1 << 24) || N < 1 || N > (1 << 20)) return invalid("M must be in [1, 2^24] and N in [1, 2^20]");
    if (K < 16 || K > 65536 || K % 16) return invalid("K must be a multiple of 16 in [16, 65536]");
    if (E < 1 || E > 4096 || (!offsets && E != 1)) return invalid("E must be in [1, 4096], and 1 without offsets");
    if ((int64_t)E * N > 0x7fffffff) return invalid("E * N must be below 2^31");
    if ((bits(a) & 15) || (bits(w) & 15)) return invalid("a and w must be 16-byte aligned");
    if ((bits(a_scale) & 3) || (bits(w_scale) & 3) || (bits(offsets) & 3) || (bits(y) & (dtype_bytes(y_dtype) - 1)))
        return invalid("scales and offsets must be 4-byte aligned and y aligned to its element");
    const DeviceInfo &di = device_info();
    if (di.device < 0) return ZFFN_ERR_CUDA;
    Fp8Args p{};
    p.a = static_cast<const uint8_t *>(a);
    p.a_scale = a_scale;
    p.offsets = offsets;
    p.w = static_cast<const uint8_t *>(w);
    p.w_scale = w_scale;
    p.y = y;
    p.y_dtype = y_dtype;
    p.M = M; p.N = N; p.K = K; p.E = E;
    p.err = di.err_word;
    return to_status(launch_fp8_matmul(p, (cudaStream_t)stream));
}

zffn_status zffn_fp8_experts(const void *a, const float *a_scale, const int32_t *offsets, const void *Wg, const float *sg,
                             const void *Wu, const float *su, const void *Wd, const float *sd, int y_dtype, void *y,
                             int P, int H, int I, int E, void *stream) {
    if (!a || !a_scale || !Wg || !sg || !Wu || !su || !Wd || !sd || !y) return invalid("a pointer argument is NULL");
    if (!dtype_valid(y_dtype)) return invalid("unknown y_dtype");
    if (check_experts(P, H, I, E) != ZFFN_OK) return ZFFN_ERR_INVALID_ARG;
    if (!offsets && E != 1) return invalid("E must be 1 without offsets");
    if ((bits(a) | bits(Wg) | bits(Wu) | bits(Wd)) & 15) return invalid("a, Wg, Wu and Wd must be 16-byte aligned");
    if (((bits(a_scale) | bits(sg) | bits(su) | bits(sd) | bits(offsets)) & 3) || (bits(y) & (dtype_bytes(y_dtype) - 1)))
        return invalid("scales and offsets must be 4-byte aligned and y aligned to its element");
    const DeviceInfo &di = device_info();
    if (di.device < 0) return ZFFN_ERR_CUDA;
    uint8_t *base = nullptr;
    const zffn_status st = workspace_at_least(experts_bytes(P, I), &base);
    if (st != ZFFN_OK) return st;
    const F8Layout L = f8_layout(P, 1, H, I, E);
    return run_experts(static_cast<const uint8_t *>(a), a_scale, offsets, Wg, sg, Wu, su, Wd, sd, y_dtype, y, P, H, I, E,
                       base + L.h, reinterpret_cast<float *>(base + L.hs), di.err_word, (cudaStream_t)stream);
}

zffn_status zffn_moe_sort(const int32_t *expert_ids, int32_t *row_slot, int32_t *slot_row, int32_t *offsets, int T,
                          int E, int top_k, void *stream) {
    if (!expert_ids || !row_slot || !slot_row || !offsets) return invalid("a pointer argument is NULL");
    if (check_route(T, E, top_k) != ZFFN_OK) return ZFFN_ERR_INVALID_ARG;
    if ((bits(expert_ids) | bits(row_slot) | bits(slot_row) | bits(offsets)) & 3) return invalid("every pointer must be 4-byte aligned");
    if (device_info().device < 0) return ZFFN_ERR_CUDA;
    return to_status(launch_moe_sort(expert_ids, row_slot, slot_row, offsets, T, E, top_k, (cudaStream_t)stream));
}

zffn_status zffn_moe_dispatch(const void *x, int64_t row_bytes, const float *scale, int64_t scale_cols,
                              const int32_t *row_slot, const int32_t *slot_row, void *xs, float *xs_scale, int T,
                              int top_k, void *stream) {
    if (!x || !row_slot || !slot_row || !xs) return invalid("a pointer argument is NULL");
    if (check_route(T, 1, top_k) != ZFFN_OK) return ZFFN_ERR_INVALID_ARG;
    if (row_bytes < 1 || row_bytes > (1 << 20)) return invalid("row_bytes must be in [1, 2^20]");
    if (scale_cols < 0 || scale_cols > (1 << 16)) return invalid("scale_cols must be in [0, 2^16]");
    if ((scale != nullptr) != (scale_cols != 0) || (xs_scale != nullptr) != (scale_cols != 0))
        return invalid("scale and xs_scale must be NULL exactly when scale_cols is 0");
    if ((bits(row_slot) | bits(slot_row) | bits(scale) | bits(xs_scale)) & 3)
        return invalid("row_slot, slot_row and the scales must be 4-byte aligned");
    if (device_info().device < 0) return ZFFN_ERR_CUDA;
    return to_status(launch_moe_dispatch(x, row_bytes, scale, scale_cols * 4, row_slot, slot_row, xs, xs_scale, T, top_k, (cudaStream_t)stream));
}

zffn_status zffn_moe_combine(int dtype, const void *rows, const int32_t *slot_row, const float *weights, float *y, int T,
                             int H, int top_k, int accumulate, void *stream) {
    if (!dtype_valid(dtype)) return invalid("unknown dtype");
    if (!rows || !slot_row || !y) return invalid("a pointer argument is NULL");
    if (check_route(T, 1, top_k) != ZFFN_OK) return ZFFN_ERR_INVALID_ARG;
    if (H < 1 || H > 65536) return invalid("H must be in [1, 65536]");
    if ((bits(rows) & (dtype_bytes(dtype) - 1)) || ((bits(slot_row) | bits(weights) | bits(y)) & 3))
        return invalid("rows must be aligned to its element, slot_row, weights and y to 4 bytes");
    if (device_info().device < 0) return ZFFN_ERR_CUDA;
    return to_status(launch_moe_combine(dtype, rows, slot_row, weights, y, T, H, top_k, accumulate != 0, (cudaStream_t)stream));
}

zffn_status zffn_moe_combine_grad(int dtype, const float *dy, const void *rows, const int32_t *row_slot,
                                  const int32_t *slot_row, const float *weights, void *drows, float *dweights, int T,
                                  int H, int top_k, void *stream) {
    if (!dtype_valid(dtype)) return invalid("unknown dtype");
    if (!dy || !row_slot || !slot_row) return invalid("a pointer argument is NULL");
    if (!drows && !dweights) return invalid("drows and dweights are both NULL");
    if ((dweights && !rows) || (drows && !weights)) return invalid("dweights needs rows, and drows needs weights");
    if (check_route(T, 1, top_k) != ZFFN_OK) return ZFFN_ERR_INVALID_ARG;
    if (H < 1 || H > 65536) return invalid("H must be in [1, 65536]");
    if (((bits(rows) | bits(drows)) & (dtype_bytes(dtype) - 1)) ||
        ((bits(dy) | bits(row_slot) | bits(slot_row) | bits(weights) | bits(dweights)) & 3))
        return invalid("rows and drows must be aligned to their element, the others to 4 bytes");
    if (device_info().device < 0) return ZFFN_ERR_CUDA;
    return to_status(launch_moe_combine_grad(dtype, dy, rows, row_slot, slot_row, weights, drows, dweights, T, H, top_k, (cudaStream_t)stream));
}

zffn_status zffn_moe_swiglu_fp8(const void *x, const int32_t *expert_ids, const float *expert_weights, const void *Wg,
                                const float *sg, const void *Wu, const float *su, const void *Wd, const float *sd,
                                float *y, int T, int H, int I, int E, int top_k, int accumulate, void *stream) {
    if (!x || !expert_ids || !expert_weights || !Wg || !sg || !Wu || !su || !Wd || !sd || !y)
        return invalid("a pointer argument is NULL");
    if (check_route(T, E, top_k) != ZFFN_OK || check_experts((int64_t)T * top_k, H, I, E) != ZFFN_OK)
        return ZFFN_ERR_INVALID_ARG;
    if ((bits(Wg) | bits(Wu) | bits(Wd)) & 15) return invalid("Wg, Wu and Wd must be 16-byte aligned");
    if ((bits(x) & 1) || ((bits(expert_ids) | bits(expert_weights) | bits(sg) | bits(su) | bits(sd) | bits(y)) & 3))
        return invalid("x must be 2-byte, and expert_ids, expert_weights, scales and y 4-byte aligned");
    const DeviceInfo &di = device_info();
    if (di.device < 0) return ZFFN_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    const int P = T * top_k;
    const F8Layout L = f8_layout(P, T, H, I, E);
    uint8_t *base = nullptr;
    zffn_status st = workspace_at_least(L.total, &base);
    if (st != ZFFN_OK) return st;
    int32_t *row_slot = reinterpret_cast<int32_t *>(base + L.row_slot), *slot_row = reinterpret_cast<int32_t *>(base + L.slot_row);
    int32_t *offsets = reinterpret_cast<int32_t *>(base + L.offsets);
    float *qs = reinterpret_cast<float *>(base + L.qs), *xs = reinterpret_cast<float *>(base + L.xs);
    cudaError_t e = launch_fp8_quantize(ZFFN_DT_BF16, x, base + L.q, qs, T, H, 1, s);
    if (e == cudaSuccess) e = launch_moe_sort(expert_ids, row_slot, slot_row, offsets, T, E, top_k, s);
    if (e == cudaSuccess)
        e = launch_moe_dispatch(base + L.q, H, qs, f8_blocks(H) * 4, row_slot, slot_row, base + L.xq, xs, T, top_k, s);
    if (e != cudaSuccess) return to_status(e);
    st = run_experts(base + L.xq, xs, offsets, Wg, sg, Wu, su, Wd, sd, ZFFN_DT_BF16, base + L.rows, P, H, I, E, base + L.h,
                     reinterpret_cast<float *>(base + L.hs), di.err_word, s);
    if (st != ZFFN_OK) return st;
    return to_status(launch_moe_combine(ZFFN_DT_BF16, base + L.rows, slot_row, expert_weights, y, T, H, top_k, accumulate != 0, s));
}

}  // extern "C"
