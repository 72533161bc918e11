// roles.cuh -- what the kernels with a role for each warp share beyond
// zffn_internal.cuh: waits that do not suspend, cluster barriers, TMA prefetches and
// stores, and the host side's encoder of tensor maps.
#pragma once

#include <cudaTypedefs.h>

#include "zffn_internal.cuh"

namespace zffn {

__device__ __forceinline__ void st_cluster_f4(uint32_t addr, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Bring a tile of a tensor map's matrix into L2.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap *map, int c0, int c1) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1)
                 : "memory");
}
// 2-D TMA tile store shared -> global, tracked by the issuing thread's bulk-async group.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, uint32_t smem_src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_src), "r"(c0), "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void named_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Whether the barrier's phase is complete, without suspending the thread.
__device__ __forceinline__ bool bar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// mbar_wait of the products' roles: the barrier is asked without suspending the
// thread (a suspended thread is woken hundreds of clocks late, once for every
// K block on the way from the tensor cores to the sums and back), and the bound
// is a count of tries: the roles have no registers to spare for the clock.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, volatile int *abort, int *err) {
    for (int n = 0; !bar_test(bar, parity); ++n)
        if (n > (1 << 26) || ((n & 1023) == 1023 && *abort)) {
            record_error(err, ZFFN_ERR_TIMEOUT);
            *abort = 1;
            return false;
        }
    return true;
}

// The same for a full warp, whose lanes all ask (one lane's answer would have to be passed on,
// which the stages wait for).
__device__ __forceinline__ bool bar_wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort, int *err) {
    return __all_sync(0xffffffffu, bar_wait(bar, parity, abort, err));
}

// The driver's encoder of tensor maps, looked up once (nullptr without one).
inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

}  // namespace zffn
