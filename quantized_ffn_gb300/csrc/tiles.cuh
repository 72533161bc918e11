// tiles.cuh -- bf16 tiles of the 5th-generation tensor cores: copies of 3-D and 4-D
// tensors, descriptors of operands as they lie in memory, tensor maps.
#pragma once

#include "roles.cuh"

namespace zffn {

constexpr int KB = 64;            // contracted values of a stage: rows of 128 bytes, or 64 rows

// 3-D TMA tile load, completion counted on `bar`.
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, uint32_t src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// Shared-memory matrix descriptor of an MN-major operand, 128-byte swizzle: boxes of 64
// values of the free index (128 bytes) by 64 (or 16, or 32) of the contracted one, box_bytes
// each; groups of 8 of the contracted index lie 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t box_bytes) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(box_bytes >> 4) << 16;     // from box to box
    d |= (uint64_t)(1024 >> 4) << 32;          // from 8 contracted values to the next
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
// Instruction descriptor: A = B = bf16, D = fp32.
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}
// What 16 contracted values are in units of a descriptor's address.
__device__ __forceinline__ uint64_t k_step(bool mn) { return mn ? 16 * 128 / 16 : 32 / 16; }
__device__ __forceinline__ uint32_t bf16x2(uint32_t lo, uint32_t hi) {
    const __nv_bfloat162 two = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
    return *reinterpret_cast<const uint32_t *>(&two);
}

// bf16 or fp32 tensor [d2][d1][d0] in boxes of 128 bytes x box1, 128-byte swizzle; loads
// give zeros past each edge, stores write nothing there.  boxes > 0: rows of a multiple of
// 64 bf16 values, of which a copy takes `boxes` boxes side by side, one after another:
// [d2][d0 / 64][d1][64].
inline bool encode(CUtensorMap *m, const void *base, int elem, int64_t d0, int64_t d1, int64_t d2, int box1, bool three, int boxes = 0) {
    cuuint64_t dims[4] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2, 1};
    cuuint64_t strides[3] = {(cuuint64_t)(d0 * elem), (cuuint64_t)(d0 * d1 * elem), 0};
    cuuint32_t box[4] = {(cuuint32_t)(128 / elem), (cuuint32_t)box1, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    cuuint32_t rank = three ? 3 : 2;
    if (boxes) {
        dims[0] = 64; dims[2] = (cuuint64_t)(d0 / 64); dims[3] = (cuuint64_t)d2;
        strides[2] = strides[1]; strides[1] = 128;
        box[2] = (cuuint32_t)boxes;
        ++rank;
    }
    return encode_fn()(m, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, rank,
                       const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace zffn
