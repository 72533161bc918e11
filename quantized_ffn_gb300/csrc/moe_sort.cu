// moe_sort.cu -- (token, slot) pairs sorted by expert, tokens' rows to their
// sorted places and the weighted sum back, and the gradients of both.
#include "moe_sort.h"

#include <atomic>

#include "launch.cuh"

namespace zffn {

namespace {

// ---------------------------------------------------------------------------
// Sort: a stable counting sort.  Every warp owns a contiguous run of pairs and
// a histogram over experts of its own; a pair's row is
//   rows of lower experts + this expert's pairs of lower warps + those before it
//   in its own warp's run,
// so no atomics decide an order and the result is the same every time.  One
// launch: a cluster of CTAs shares the warps' totals through distributed
// shared memory.  Latency bound (16 bytes a pair move): 32768 pairs take 6.3 us,
// 262144 on the same 16 CTAs 25.4 us.
// ---------------------------------------------------------------------------
constexpr int kSortMaxWarps = 32;      // of one CTA alone; 16 of a cluster's (a turn of 32 pairs costs a
constexpr int kSortClusterWarps = 16;  // warp about 0.6 us, so 32768 pairs took 6.8 us on 16 x 16 warps,
constexpr int kSortCluster = 16;       // 9.8 us on 8 x 32 and 12.7 us there with the count by matches)

__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Shared memory: hist [warps][E], total [E] (this CTA's pairs of each expert),
// base [E], 33 words of scan scratch.
constexpr int kSortKeys = 8;   // turns of a warp whose keys stay in registers from the count to the placing

template <int CS>
__global__ void __launch_bounds__(kSortMaxWarps * 32)
    moe_sort_kernel(const int32_t *__restrict__ ids, int32_t *__restrict__ row_slot, int32_t *__restrict__ slot_row,
                    int32_t *__restrict__ offsets, int P, int E) {
    extern __shared__ int sm[];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int *hist = sm, *total = sm + warps * E, *base = total + E, *scratch = base + E;
    const int rank = CS > 1 ? (int)cluster_ctarank() : 0;
    grid_wait();
    grid_launch_dependents();
    // this warp's run of pairs, a multiple of 32 long
    const int64_t all = (int64_t)CS * warps;
    const int64_t run = ((P + all - 1) / all + 31) / 32 * 32;
    const int64_t lo = ((int64_t)rank * warps + warp) * run;
    const int64_t hi = lo + run < P ? lo + run : P;
    auto load_key = [&](int64_t i) {
        const int e = i < hi ? __ldg(ids + i) : -1;
        return e < 0 || e >= E ? -1 : e;
    };
    int key[kSortKeys];
#pragma unroll
    for (int k = 0; k < kSortKeys; ++k) key[k] = load_key(lo + 32 * k + lane);
    for (int i = threadIdx.x; i < warps * E; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    int *mine = hist + warp * E;
    auto count = [&](int e) {   // (a sum: the order of the additions does not show)
        if (e >= 0) atomicAdd(&mine[e], 1);
    };
#pragma unroll
    for (int k = 0; k < kSortKeys; ++k)
        if (lo + 32 * k < hi) count(key[k]);
    for (int64_t i = lo + 32 * kSortKeys; i < hi; i += 32) count(load_key(i + lane));
    __syncthreads();
    // each expert: exclusive sums over this CTA's warps, and the CTA's total
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int c[kSortMaxWarps], n = 0;
#pragma unroll
        for (int w = 0; w < kSortMaxWarps; ++w) c[w] = w < warps ? hist[w * E + e] : 0;
#pragma unroll
        for (int w = 0; w < kSortMaxWarps; ++w) {
            if (w < warps) hist[w * E + e] = n;
            n += c[w];
        }
        total[e] = n;
    }
    if (CS > 1) cluster_sync_all();
    else __syncthreads();
    // over the cluster: the expert's pairs in all CTAs (base, scanned below) and
    // in the CTAs before this one
    const uint32_t t_addr = smem_u32(total);
    const int per = (E + blockDim.x - 1) / blockDim.x;   // experts of a thread, consecutive
    const int e0 = threadIdx.x * per, e1 = min(E, e0 + per);
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
        int n = total[e];
        if (CS > 1) {
            int c[CS], before = 0;
#pragma unroll
            for (int r = 0; r < CS; ++r) c[r] = ld_cluster_s32(mapa_shared(t_addr + 4 * e, r));
            n = 0;
#pragma unroll
            for (int r = 0; r < CS; ++r) {
                if (r < rank) before += c[r];
                n += c[r];
            }
            base[e] = before;
        }
        sum += n;
        // (total is still read by other CTAs: n is summed up again below)
    }
    // exclusive scan over the threads' shares
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
    }
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const int wt = lane < warps ? scratch[lane] : 0;
        int winc = wt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, winc, o);
            if (lane >= o) winc += t;
        }
        scratch[lane] = winc - wt;
        if (lane == 31) scratch[32] = winc;
    }
    __syncthreads();
    int at = scratch[warp] + inc - sum;
    for (int e = e0; e < e1; ++e) {
        int n = per == 1 ? sum : total[e];
        if (CS > 1 && per > 1) {
            n = 0;
#pragma unroll
            for (int r = 0; r < CS; ++r) n += ld_cluster_s32(mapa_shared(t_addr + 4 * e, r));
        }
        base[e] = at + (CS > 1 ? base[e] : 0);   // this CTA's first row of the expert
        if (rank == 0) offsets[e] = at;
        at += n;
    }
    // the other CTAs' totals have been read: this is waited for before leaving
    if (CS > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    const int used = scratch[32];
    if (rank == 0 && threadIdx.x == 0) offsets[E] = used;
    __syncthreads();
    auto place = [&](int64_t i, int e) {
        const unsigned same = __match_any_sync(0xffffffffu, e);
        int row = -1;
        if (e >= 0) row = base[e] + mine[e] + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
        if (i < hi) {
            slot_row[i] = row;
            // a row from `used` on is nobody's: its own index is as good a place as any
            if (i >= used) row_slot[i] = -1;
        }
        if (row >= 0) row_slot[row] = (int)i;
    };
#pragma unroll
    for (int k = 0; k < kSortKeys; ++k)
        if (lo + 32 * k < hi) place(lo + 32 * k + lane, key[k]);
    for (int64_t i = lo + 32 * kSortKeys; i < hi; i += 32) place(i + lane, load_key(i + lane));
    if (CS > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Rows to their sorted places.  A thread block per token and share of its row,
// which is read once and written to each of its places.  Bound by HBM writes: 32768
// rows of 4 KB (8 of each token) take 25.5 us, 5.9 TB/s.
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 128;

// Steps that a thread takes at once, kRowThreads apart: one of 16 bytes, four of
// less (rows that are not 16-byte multiples), to have as much in flight.
template <int BYTES> constexpr int kRowSteps = BYTES >= 16 ? 1 : 4;

template <typename V>
__device__ __forceinline__ void copy_row(const V *__restrict__ src, V *__restrict__ dst, int64_t n, int64_t P,
                                         const int32_t *rows, const int32_t *row_slot, int64_t t, int k) {
    constexpr int U = kRowSteps<sizeof(V)>;
    for (int64_t c = (int64_t)blockIdx.y * kRowThreads * U + threadIdx.x; c < n; c += (int64_t)gridDim.y * kRowThreads * U) {
        V v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u * kRowThreads < n) v[u] = __ldg(src + t * n + c + u * kRowThreads);
        for (int j = 0; j < k; ++j) {
            const int64_t r = rows[j];
            if (r < 0 || r >= P) continue;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c + u * kRowThreads < n) dst[r * n + c + u * kRowThreads] = v[u];
        }
    }
    // rows of no pair: block t looks after rows t k .. t k + k - 1
    for (int j = 0; j < k; ++j) {
        const int64_t r = t * k + j;
        if (row_slot[r] >= 0) continue;
        for (int64_t c = blockIdx.y * kRowThreads + threadIdx.x; c < n; c += gridDim.y * kRowThreads) dst[r * n + c] = V{};
    }
}

template <typename V>
__global__ void __launch_bounds__(kRowThreads)
    moe_dispatch_kernel(const V *__restrict__ x, int64_t n, const uint32_t *__restrict__ scale, int64_t ns,
                        const int32_t *__restrict__ row_slot, const int32_t *__restrict__ slot_row, V *__restrict__ xs,
                        uint32_t *__restrict__ xs_scale, int T, int k) {
    __shared__ int32_t rows[64];
    grid_wait();
    grid_launch_dependents();
    const int64_t t = blockIdx.x, P = (int64_t)T * k;
    if ((int)threadIdx.x < k) rows[threadIdx.x] = slot_row[t * k + threadIdx.x];
    __syncthreads();
    copy_row(x, xs, n, P, rows, row_slot, t, k);
    if (ns) copy_row(scale, xs_scale, ns, P, rows, row_slot, t, k);
}

// ---------------------------------------------------------------------------
// Vectors of the row type: VEC elements as fp32.
// ---------------------------------------------------------------------------
template <int VEC> struct Vec { float v[VEC]; };

// The same as it lies in memory.
template <typename T, int VEC> struct Raw;
template <> struct Raw<__nv_bfloat16, 8> { uint4 a; };
template <> struct Raw<__nv_bfloat16, 2> { uint32_t a; };
template <> struct Raw<__nv_bfloat16, 1> { uint32_t a; };   // (a register each: halves of one would wait for each other)
template <> struct Raw<float, 8> { uint4 a, b; };
template <> struct Raw<float, 2> { uint2 a; };
template <> struct Raw<float, 1> { uint32_t a; };

template <typename T, int VEC> __device__ __forceinline__ Raw<T, VEC> load_raw(const T *p) {
    Raw<T, VEC> r;
    if constexpr (sizeof(T) * VEC == 2) r.a = __ldg(reinterpret_cast<const uint16_t *>(p));
    else r.a = __ldg(reinterpret_cast<const decltype(r.a) *>(p));
    if constexpr (sizeof(T) * VEC == 32) r.b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    return r;
}
template <int VEC> __device__ __forceinline__ Vec<VEC> unpack(const Raw<__nv_bfloat16, VEC> &r) {
    Vec<VEC> v;
    if constexpr (VEC == 8) {
        const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v.v[2 * i] = __uint_as_float(w[i] << 16);
            v.v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else if constexpr (VEC == 2) {
        v.v[0] = __uint_as_float(r.a << 16);
        v.v[1] = __uint_as_float(r.a & 0xFFFF0000u);
    } else {
        v.v[0] = __uint_as_float(r.a << 16);
    }
    return v;
}
template <int VEC> __device__ __forceinline__ Vec<VEC> unpack(const Raw<float, VEC> &r) {
    Vec<VEC> v;
    if constexpr (VEC == 8) {
        const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v.v[i] = __uint_as_float(w[i]);
    } else if constexpr (VEC == 2) {
        v.v[0] = __uint_as_float(r.a.x);
        v.v[1] = __uint_as_float(r.a.y);
    } else {
        v.v[0] = __uint_as_float(r.a);
    }
    return v;
}
// A bf16 value of row r, column c; zero where r < 0 or c >= H.  (Loaded from a place
// within the rows in any case and then chosen: with a test before it each such
// load waited for the one before.)
__device__ __forceinline__ Raw<__nv_bfloat16, 1> load_one(const __nv_bfloat16 *rows, int r, int c, int H) {
    Raw<__nv_bfloat16, 1> x = load_raw<__nv_bfloat16, 1>(rows + (int64_t)max(r, 0) * H + min(c, H - 1));
    if (r < 0 || c >= H) x.a = 0;
    return x;
}
template <int VEC, typename T> __device__ __forceinline__ Vec<VEC> load_vec(const T *p) { return unpack<VEC>(load_raw<T, VEC>(p)); }
template <int VEC> __device__ __forceinline__ void store_vec(float *p, const Vec<VEC> &r) {
    if (VEC == 8) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i)
            reinterpret_cast<float4 *>(p)[i] = make_float4(r.v[4 * i], r.v[4 * i + 1], r.v[4 * i + 2], r.v[4 * i + 3]);
    } else if (VEC == 2) {
        *reinterpret_cast<float2 *>(p) = make_float2(r.v[0], r.v[VEC - 1]);
    } else {
        p[0] = r.v[0];
    }
}
// (one rounding to bf16, to nearest even)
template <int VEC> __device__ __forceinline__ void store_vec(__nv_bfloat16 *p, const Vec<VEC> &r) {
    if (VEC == 8) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(r.v[2 * i], r.v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if (VEC == 2) {
        *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(r.v[0], r.v[VEC - 1]);
    } else {
        p[0] = __float2bfloat16_rn(r.v[0]);
    }
}

// ---------------------------------------------------------------------------
// Sorted rows back to tokens: a thread block per token and share of its columns,
// fp32 sums over the slots in order.  Bound by HBM reads: 32768 rows of 2048 bf16
// to 4096 of fp32 take 26.8 us, 6.3 TB/s.
// ---------------------------------------------------------------------------
template <typename T, int VEC>
__global__ void __launch_bounds__(kRowThreads, VEC == 8 ? 12 : 8)   // (registers for the loads in flight: without it 31 us)
    moe_combine_kernel(const T *__restrict__ rows, const int32_t *__restrict__ slot_row, const float *__restrict__ weights,
                       float *__restrict__ y, int Tn, int H, int k, bool accumulate) {
    __shared__ int32_t row[64];
    __shared__ float wt[64];
    grid_wait();
    grid_launch_dependents();
    const int64_t t = blockIdx.x, P = (int64_t)Tn * k;
    if ((int)threadIdx.x < k) {
        const int r = slot_row[t * k + threadIdx.x];
        const bool some = r >= 0 && r < P;
        row[threadIdx.x] = some ? r : -1;
        wt[threadIdx.x] = some ? (weights ? weights[t * k + threadIdx.x] : 1.0f) : 0.0f;
    }
    __syncthreads();
    constexpr int U = kRowSteps<VEC * (int)sizeof(T)>, APART = kRowThreads * VEC;
    for (int c = blockIdx.y * APART * U + threadIdx.x * VEC; c < H; c += gridDim.y * APART * U) {
        Vec<VEC> acc[U];
        float *py = y + t * H + c;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[u].v[i] = accumulate && c + u * APART < H ? py[u * APART + i] : 0.0f;
        // SLOTS slots at a time, their loads before their sums (pairs without a row: zero
        // times zero): 32768 rows of 2048 bf16 26.9 us, with a load, a test and a sum in
        // turn 30.2 us
        constexpr int SLOTS = U == 1 ? 128 / (VEC * (int)sizeof(T)) : VEC * (int)sizeof(T) == 8 ? 4 : 8;
        for (int j0 = 0; j0 < k; j0 += SLOTS) {
            Raw<T, VEC> x[SLOTS][U];
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                const int r = j0 + j < k ? row[j0 + j] : -1;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if constexpr (sizeof(T) * VEC == 2) {
                        x[j][u] = load_one(rows, r, c + u * APART, H);
                    } else {
                        x[j][u] = Raw<T, VEC>{};
                        if (r >= 0 && c + u * APART < H) x[j][u] = load_raw<T, VEC>(rows + (int64_t)r * H + c + u * APART);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                const float w = j0 + j < k ? wt[j0 + j] : 0.0f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const Vec<VEC> v = unpack<VEC>(x[j][u]);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) acc[u].v[i] = fmaf(w, v.v[i], acc[u].v[i]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u * APART < H) store_vec<VEC>(py + u * APART, acc[u]);
    }
}

// ---------------------------------------------------------------------------
// Gradients of the combine: a warp per (token, slot); the token's dy row is
// shared by the block's warps through L1.  Bound by HBM: 32768 rows of 2048 bf16
// take 48 us, 6.3 TB/s.
// ---------------------------------------------------------------------------
constexpr int kGradWarps = 8;

template <typename T, int VEC>
__global__ void __launch_bounds__(kGradWarps * 32, VEC == 8 ? 4 : 0)
    moe_combine_grad_kernel(const float *__restrict__ dy, const T *__restrict__ rows, const int32_t *__restrict__ row_slot,
                            const int32_t *__restrict__ slot_row, const float *__restrict__ weights,
                            T *__restrict__ drows, float *__restrict__ dweights, int Tn, int H, int k) {
    grid_wait();
    grid_launch_dependents();
    const int64_t t = blockIdx.x, P = (int64_t)Tn * k;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float *d = dy + t * H;
    for (int j = warp; j < k; j += kGradWarps) {
        const int64_t f = t * k + j;
        const int64_t r = slot_row[f];
        if (r >= 0 && r < P) {
            const float w = drows ? weights[f] : 0.0f;
            float dot = 0.0f;
            // STEPS steps of the row at a time, their loads first
            constexpr int STEPS = VEC == 8 ? 2 : 8;
            for (int c = lane * VEC; c < H; c += 32 * VEC * STEPS) {
                Raw<float, VEC> g[STEPS];
                Raw<T, VEC> x[STEPS];
#pragma unroll
                for (int u = 0; u < STEPS; ++u) {
                    g[u] = Raw<float, VEC>{};
                    x[u] = Raw<T, VEC>{};
                    const int at = c + u * 32 * VEC;
                    if constexpr (sizeof(T) * VEC == 2) {
                        if (at < H) g[u] = load_raw<float, VEC>(d + at);
                        if (dweights) x[u] = load_one(rows, (int)r, at, H);
                    } else if (at < H) {
                        g[u] = load_raw<float, VEC>(d + at);
                        if (dweights) x[u] = load_raw<T, VEC>(rows + r * H + at);
                    }
                }
#pragma unroll
                for (int u = 0; u < STEPS; ++u) {
                    const int at = c + u * 32 * VEC;
                    const Vec<VEC> gv = unpack<VEC>(g[u]), v = unpack<VEC>(x[u]);
                    Vec<VEC> o;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        dot = fmaf(gv.v[i], v.v[i], dot);
                        o.v[i] = w * gv.v[i];
                    }
                    if (drows && at < H) store_vec<VEC>(drows + r * H + at, o);
                }
            }
            if (dweights) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                if (lane == 0) dweights[f] = dot;
            }
        } else if (dweights && lane == 0) {
            dweights[f] = 0.0f;
        }
        // row f itself, where no pair has it
        if (drows && row_slot[f] < 0) {
            Vec<VEC> o;
#pragma unroll
            for (int i = 0; i < VEC; ++i) o.v[i] = 0.0f;
            for (int c = lane * VEC; c < H; c += 32 * VEC) store_vec<VEC>(drows + f * H + c, o);
        }
    }
}

inline uintptr_t bits(const void *p) { return reinterpret_cast<uintptr_t>(p); }

// Blocks of a token of n column steps, `steps` a thread; at most 16.
inline dim3 row_grid(int T, int64_t n, int steps) {
    const int64_t y = (n + kRowThreads * steps - 1) / (kRowThreads * steps);
    return dim3((unsigned)T, (unsigned)(y < 16 ? y : 16));
}

template <typename V>
cudaError_t dispatch_as(const void *x, int64_t row_bytes, const void *scale, int64_t scale_bytes,
                        const int32_t *row_slot, const int32_t *slot_row, void *xs, void *xs_scale, int T, int k,
                        cudaStream_t s) {
    const int64_t n = row_bytes / (int64_t)sizeof(V);
    return launch_dependent(moe_dispatch_kernel<V>, row_grid(T, n, kRowSteps<sizeof(V)>), kRowThreads, 0, 1, s, static_cast<const V *>(x), n,
                            static_cast<const uint32_t *>(scale), scale_bytes / 4, row_slot, slot_row, static_cast<V *>(xs),
                            static_cast<uint32_t *>(xs_scale), T, k);
}

template <typename T>
cudaError_t combine_as(const T *rows, const int32_t *slot_row, const float *weights, float *y, int Tn, int H, int k,
                       bool accumulate, cudaStream_t s) {
    auto run = [&](auto kernel, int vec, int steps) {
        return launch_dependent(kernel, row_grid(Tn, H / vec, steps), kRowThreads, 0, 1, s, rows, slot_row, weights, y, Tn, H, k, accumulate);
    };
    constexpr int E = (int)sizeof(T);
    if (((bits(rows) | bits(y)) & 15) == 0 && H % 8 == 0) return run(moe_combine_kernel<T, 8>, 8, kRowSteps<8 * E>);
    if ((bits(rows) & (2 * E - 1)) == 0 && (bits(y) & 7) == 0 && H % 2 == 0) return run(moe_combine_kernel<T, 2>, 2, kRowSteps<2 * E>);
    return run(moe_combine_kernel<T, 1>, 1, kRowSteps<E>);
}

template <typename T>
cudaError_t grad_as(const float *dy, const T *rows, const int32_t *row_slot, const int32_t *slot_row,
                    const float *weights, T *drows, float *dweights, int Tn, int H, int k, cudaStream_t s) {
    auto run = [&](auto kernel) {
        return launch_dependent(kernel, dim3(Tn), kGradWarps * 32, 0, 1, s, dy, rows, row_slot, slot_row, weights, drows, dweights, Tn, H, k);
    };
    constexpr int E = (int)sizeof(T);
    if (((bits(dy) | bits(rows) | bits(drows)) & 15) == 0 && H % 8 == 0) return run(moe_combine_grad_kernel<T, 8>);
    if (((bits(rows) | bits(drows)) & (2 * E - 1)) == 0 && (bits(dy) & 7) == 0 && H % 2 == 0) return run(moe_combine_grad_kernel<T, 2>);
    return run(moe_combine_grad_kernel<T, 1>);
}

}  // namespace

cudaError_t launch_moe_sort(const int32_t *ids, int32_t *row_slot, int32_t *slot_row, int32_t *offsets,
                            int T, int E, int k, cudaStream_t s) {
    const int64_t P = (int64_t)T * k;
    // as many warps as their histograms fit into 160 KB (E = 4096: 10), and no
    // more than the pairs fill
    int warps = (160 * 1024) / (4 * E);
    if (warps > kSortMaxWarps) warps = kSortMaxWarps;
    const bool one = P <= 32 * kSortMaxWarps;
    // (one CTA: enough warps for the pairs, and for a thread to an expert in the scan)
    const int64_t need = (P + 31) / 32 > (E + 31) / 32 ? (P + 31) / 32 : (E + 31) / 32;
    if (one && warps > need) warps = (int)need;
    if (!one && warps > kSortClusterWarps) warps = kSortClusterWarps;
    const int smem = 4 * ((warps + 2) * E + 33);
    const void *fn = one ? (const void *)moe_sort_kernel<1> : (const void *)moe_sort_kernel<kSortCluster>;
    const cudaError_t e = ensure_dynamic_smem(fn, (size_t)smem);
    if (e != cudaSuccess) return e;
    if (one) {
        return launch_dependent(moe_sort_kernel<1>, dim3(1), warps * 32, smem, 1, s, ids, row_slot, slot_row, offsets, P, E);
    }
    // clusters of more than 8 CTAs have to be asked for, once a device
    static std::atomic<uint64_t> allowed{0};
    const uint64_t bit = 1ull << (device_info().device & 63);
    if (!(allowed.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t a = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (a != cudaSuccess) return a;
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_dependent(moe_sort_kernel<kSortCluster>, dim3(kSortCluster), warps * 32, smem, kSortCluster, s, ids, row_slot, slot_row,
                            offsets, P, E);
}

cudaError_t launch_moe_dispatch(const void *x, int64_t row_bytes, const void *scale, int64_t scale_bytes,
                                const int32_t *row_slot, const int32_t *slot_row, void *xs, void *xs_scale,
                                int T, int k, cudaStream_t s) {
    const uintptr_t a = bits(x) | bits(xs) | (uintptr_t)row_bytes;   // the widest copy that every row allows
    if ((a & 15) == 0) return dispatch_as<uint4>(x, row_bytes, scale, scale_bytes, row_slot, slot_row, xs, xs_scale, T, k, s);
    if ((a & 7) == 0) return dispatch_as<uint2>(x, row_bytes, scale, scale_bytes, row_slot, slot_row, xs, xs_scale, T, k, s);
    if ((a & 3) == 0) return dispatch_as<uint32_t>(x, row_bytes, scale, scale_bytes, row_slot, slot_row, xs, xs_scale, T, k, s);
    if ((a & 1) == 0) return dispatch_as<uint16_t>(x, row_bytes, scale, scale_bytes, row_slot, slot_row, xs, xs_scale, T, k, s);
    return dispatch_as<uint8_t>(x, row_bytes, scale, scale_bytes, row_slot, slot_row, xs, xs_scale, T, k, s);
}

cudaError_t launch_moe_combine(int dtype, const void *rows, const int32_t *slot_row, const float *weights,
                               float *y, int T, int H, int k, bool accumulate, cudaStream_t s) {
    if (dtype == ZFFN_DT_F32)
        return combine_as(static_cast<const float *>(rows), slot_row, weights, y, T, H, k, accumulate, s);
    return combine_as(static_cast<const __nv_bfloat16 *>(rows), slot_row, weights, y, T, H, k, accumulate, s);
}

cudaError_t launch_moe_combine_grad(int dtype, const float *dy, const void *rows, const int32_t *row_slot,
                                    const int32_t *slot_row, const float *weights, void *drows,
                                    float *dweights, int T, int H, int k, cudaStream_t s) {
    if (dtype == ZFFN_DT_F32)
        return grad_as(dy, static_cast<const float *>(rows), row_slot, slot_row, weights, static_cast<float *>(drows),
                       dweights, T, H, k, s);
    return grad_as(dy, static_cast<const __nv_bfloat16 *>(rows), row_slot, slot_row, weights,
                   static_cast<__nv_bfloat16 *>(drows), dweights, T, H, k, s);
}

}  // namespace zffn
