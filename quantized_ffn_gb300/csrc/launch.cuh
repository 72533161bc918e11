// launch.cuh -- what the 8-bit and sorting entry points share beyond
// zffn_internal.cuh: the host side's checks and workspace (defined in api.cu), and
// programmatic launches.
#pragma once

#include "zffn_internal.cuh"

namespace zffn {

// A failed host-side check: record why (zffn_last_error) and return INVALID_ARG.
zffn_status invalid(const char *why);
// A CUDA status as the library's; an error is recorded for zffn_last_error.
zffn_status to_status(cudaError_t e);
// The current device's workspace, grown to at least `bytes`.  Its first 256 bytes
// belong to the one-launch routed path (a count that outlives a call).
zffn_status workspace_at_least(size_t bytes, uint8_t **base);
// Workspace of the block-scaled 8-bit entry points for calls up to these sizes.
size_t fp8_workspace_bytes(int T, int H, int I, int E, int k);

// ---------------------------------------------------------------------------
// Programmatic launches: the kernel may be scheduled while the grid before it in
// the stream ends, and waits for it (grid_wait) before it touches anything of the
// caller's; it lets the next grid be scheduled in turn (grid_launch_dependents).
// ---------------------------------------------------------------------------
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// (cluster > 1: a cluster launch)
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, unsigned cluster,
                                    cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace zffn
