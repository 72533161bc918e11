// fp8_matmul.cu -- products of block-scaled e4m3 matrices on the 5th-generation
// tensor cores, dense or grouped by expert, plain or with SwiGLU and
// quantisation of the result:
//     y[m][n] = sum_b sa[m][b] sw[n/128][b] sum_{k in block b} a[m][k] w[n][k]
// The scales are any fp32 values, so a block's product (K = 128, four MMAs of
// K = 32) is one accumulation in tensor memory, and the sum over blocks is kept
// in registers: acc += d * (sa * sw), one fp32 multiply-add per value and block
// (the scales' product is rounded once before; below 2^-126 it is held in steps of
// 2^-149, which moves a block's term by less than 2^-125, since its sum is below 2^25).
#include <atomic>

#include "fp8.h"
#include "launch.cuh"
#include "roles.cuh"

namespace zffn {
namespace f8 {

// ---- pieces -----------------------------------------------------------------

// D[tmem] (+)= A[smem desc] * B[smem desc]^T, e4m3 inputs, fp32 accumulate.
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// The same over a CTA pair: D in both CTAs' tensor memory, A from both, B split between them.
__device__ __forceinline__ void tc_mma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Instruction descriptor: A = B = e4m3 (format code 0), D = fp32, both K-major.
__host__ __device__ constexpr uint32_t idesc_f8_f32(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// acc += d * s on a pair of fp32 values (one instruction, each half rounded once).
__device__ __forceinline__ void fma2(float2 &acc, uint32_t d0, uint32_t d1, float s0, float s1) {
    asm("{\n\t.reg .b64 a, d, f;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 d, {%2, %3};\n\tmov.b64 f, {%4, %5};\n\t"
        "fma.rn.f32x2 a, d, f, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(acc.x), "+f"(acc.y)
        : "r"(d0), "r"(d1), "f"(s0), "f"(s1));
}
__device__ __forceinline__ void fma2(float2 &acc, uint32_t d0, uint32_t d1, float s) { fma2(acc, d0, d1, s, s); }
template <int N> struct Bytes { static constexpr int value = N; };
template <int R> __device__ __forceinline__ void reg_alloc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R> __device__ __forceinline__ void reg_dealloc() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
// silu(g) u = g / (1 + 2^(-g log2 e)) u: two instructions of the special function
// unit and four others.  Off by at most (3 + |g| / 3) 2^-22 of the value for g < 0
// and 3 x 2^-22 for g > 0: the exponent -g log2 e is rounded to fp32, by up to 2^-24
// of itself and the constant by 2^-26, and the instructions are off by 2^-22 and 2^-23
// (with exact ones 1.4 x 2^-22 at g = -5, 8 at -40, 16 at -87), where h keeps 2^-4.
// Below g = -87.3 the reciprocal is subnormal and h is 0; silu is above -1.1e-36
// there.  Written out once for each value that a thread
// holds, so its length counts: with the divide's and exponential's own handling of
// denormals a 128 x 128 tile of h took 7500 clocks, fetching instructions.
__device__ __forceinline__ float swiglu(float g, float u) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return g * r * u;
}

struct Params {
    const float *sa, *sw0, *sw1;
    const int32_t *offsets;
    void *y;
    float *y_scale;
    int *err;
    int M, N, K, E;
    int row_tiles;      // bound of the number of row tiles
    int n_tiles;        // large: tiles of W's rows
    int y_bf16;         // plain: y is bf16 (else fp32)
    int early;          // small: all but a and its scales are complete before the previous grid is
    int vec;            // y's rows take vector stores (small: 4 elements, large: 16 bytes)
};
struct Maps {
    CUtensorMap a, w0, w1, y;   // y: the large tiles' stores
};

// A tile of the result: rows of one expert (e == E: rows of none) times a tile of W's rows.
struct RowTile {
    int e, row0, rows, nt;
};

// Tile i of a cluster's walk: the group of rows, its rows, the W tile.
template <class C>
struct Walk {
    int e, row0, rows, nt;   // rows: of the tile, <= C::TM
    int t;

    __device__ __forceinline__ void start(int cluster) { t = cluster; e = 0; }
    // false past the last tile.  One full warp.  cum[g]: row tiles before group
    // g and its first row; one entry past the last.
    __device__ __forceinline__ bool get(const Params &p, const int2 *cum) {
        const int n_tiles = p.n_tiles;
        if (!p.offsets) {
            const int rt_all = p.row_tiles;
            if (t >= rt_all * n_tiles) return false;
            const int first = t / (C::GROUP * n_tiles) * C::GROUP;
            const int in = t - first * n_tiles, wide = min(C::GROUP, rt_all - first);
            nt = in / wide;
            row0 = (first + in - nt * wide) * C::TM;
            rows = min(C::TM, p.M - row0);
            return true;
        }
        const int groups = p.E + 1;
        if (t >= cum[groups].x * n_tiles) return false;
        const int rt = t / n_tiles, lane = threadIdx.x & 31;
        nt = t - rt * n_tiles;
        for (;; e += 32) {   // the group whose tiles hold rt: ascending from the last one
            const unsigned past = __ballot_sync(0xffffffffu, cum[min(e + lane + 1, groups)].x > rt);
            if (past) {
                e += __ffs(past) - 1;
                break;
            }
        }
        const int2 at = cum[e];
        row0 = at.y + (rt - at.x) * C::TM;
        rows = min(C::TM, (e < p.E ? cum[e + 1].y : p.M) - row0);
        return true;
    }
};

// The groups of rows (the experts, then the rows of none; h needs no zeros there)
// in shared memory: {row tiles before the group, its first row}, one entry past the
// last.  Called by the whole block.  Whatever the offsets hold, the groups part the
// rows: an offset counts as the largest of those up to it, kept within [0, M], so that
// the row tiles are never more than row_tiles_bound, which the grid is sized by.
// sums: 2 * THREADS / 32 words of shared memory that nothing else uses yet.
template <class C>
__device__ __forceinline__ void build_groups(const Params &p, int2 *cum, int *sums) {
    // a thread to a group, THREADS groups at a time: sums within the warps by shuffles,
    // over the warps through shared memory
    constexpr int WARPS = C::THREADS / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int before = 0;
    bool descend = false;
    auto offset = [&](int g) { return min(max(__ldcg(p.offsets + g), 0), p.M); };   // (from L2: an early grid reads them before its wait)
    for (int g0 = 0, half = 0; g0 <= p.E; g0 += C::THREADS, half ^= 1) {
        const int g = g0 + threadIdx.x;
        int lo = 0, hi = 0, n, inc;
        if (g <= p.E) {
            lo = offset(g);
            hi = g < p.E ? offset(g + 1) : (C::GU ? lo : p.M);
        }
        auto scan = [&] {
            n = (hi - lo + C::TM - 1) / C::TM;
            inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            if (lane == 31) sums[half * WARPS + warp] = inc;
        };
        scan();
        if (__syncthreads_or(hi < lo || descend)) {
            // (never for offsets as the sort writes them, so the running maximum is
            // found the plain way)
            descend = true;
            lo = 0;
            for (int i = 0; i <= min(g, p.E); ++i) lo = max(lo, offset(i));
            hi = g < p.E ? max(lo, offset(g + 1)) : (C::GU || g > p.E ? lo : p.M);
            scan();
            __syncthreads();
        }
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            if (w < warp) before += sums[half * WARPS + w];
        if (g <= p.E) cum[g] = make_int2(before + inc - n, lo);
        if (g == p.E) cum[p.E + 1] = make_int2(before + inc, p.M);
        if (g0 + C::THREADS <= p.E)
            for (int w = warp; w < WARPS; ++w) before += sums[half * WARPS + w];
    }
}

// ---------------------------------------------------------------------------
// Few rows an expert: the weights on the MMA's M side.  A tile is 128 rows of W
// (GU: 128 gate and 128 up rows) times TN rows of a; each cluster takes tiles in
// turn, the ring of TMA loads running on from one to the next.  Where the tiles
// are fewer than the SMs a cluster's blocks split K: row j's sums go to the shared
// memory of rank j % split, which adds them in rank order, so that the result is
// the same every time.  (Each rank writes to the others: one barrier of the
// cluster, where reading from the others takes a second one before a block may
// leave, 0.8 us.)  Bound by HBM: every weight byte is read once.  The experts of
// 256 tokens (128 of 2048 x 768, 8 a token; 617 MB) take 100 us, 6.2 TB/s.  Short
// calls are bound by the way from the launch to the first bytes and from the last
// ones through the join: 1 x 11008 x 4096 (45 MB) takes 10.1 us, 4.5 TB/s.
//
// Roles: warps 0 .. 4 NW - 1 take a block's product out of tensor memory, scale
// and sum it in registers, and write the result; then one warp loads by TMA and
// one issues the MMAs.
// ---------------------------------------------------------------------------
template <int TN_, bool GU_>
struct SmallCfg {
    static constexpr int TN = TN_, TM = TN_;
    static constexpr bool GU = GU_;
    static constexpr int CTAS = 1;
    static constexpr int TNW = 128;                          // rows of W (of each, GU)
    static constexpr int GROUP = 8;                          // dense: row tiles that share a W tile in turn
    static constexpr int NW = GU ? 2 : 1;                    // weight tiles
    static constexpr int W_BYTES = 128 * 128;
    static constexpr int STAGE = NW * W_BYTES + TN * 128;
    static constexpr int BLOCKS = GU ? 1 : 2;                // blocks an SM
    // (GU, TN = 16: three, so that a block of the down product fits beside it)
    static constexpr int NS = GU ? (TN == 32 ? 5 : 3) : TN == 64 ? 3 : 4;
    static constexpr int NB = TN == 16 ? 4 : 2;              // accumulators in tensor memory
    static constexpr int TMEM_COLS = NB * NW * TN;           // 64 .. 256, a power of two
    static constexpr int SEG = 4;                            // K blocks of scales kept at a time
    static constexpr int TAB = NW * SEG * TN;                // floats of one segment's scales
    static constexpr int EPI = 4 * NW;                       // warps that sum
    static constexpr int THREADS = (EPI + 2) * 32;
    static constexpr int MAX_SPLIT = 8;
    // sums [weight tile][rank][row / split][128]
    static constexpr int PART_ROWS = TN + MAX_SPLIT - 1;     // split * ceil(TN / split), at most
    static constexpr int OFF_PART = NS * STAGE;
    static_assert(NW * TN * 128 * 4 <= NS * STAGE, "a block's own sums fit into its ring");
    static constexpr int OFF_TAB = OFF_PART + NW * PART_ROWS * 128 * 4;
    static constexpr int OFF_BAR = OFF_TAB + 2 * TAB * 4;
    static constexpr int OFF_CUM = OFF_BAR + (2 * NS + 2 * NB + 1) * 8 + 8;
    static constexpr int SMEM = OFF_CUM + 1024;              // + {row tiles before, first row} of each group of rows
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::BLOCKS) small_kernel(const __grid_constant__ Maps maps, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float *part = reinterpret_cast<float *>(smem + C::OFF_PART);
    float *tab = reinterpret_cast<float *>(smem + C::OFF_TAB);
    uint64_t *s_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *s_empty = s_full + C::NS, *t_full = s_empty + C::NS, *t_empty = t_full + C::NB, *done = t_empty + C::NB;
    int *info = reinterpret_cast<int *>(done + 1);           // abort, TMEM base
    int2 *cum = reinterpret_cast<int2 *>(smem + C::OFF_CUM);
    volatile int *abort_flag = info;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t split;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(split));
    const uint32_t rank = cluster_ctarank();
    const uint32_t slice = (C::TN + split - 1) / split;       // rows of a tile that a rank adds up
    const uint32_t inverse = (65536 + split - 1) / split;     // j * inverse >> 16 = j / split for j < 64
    if (split > 1) cluster_arrive();                          // (waited for before another's memory is written)
    if (warp == C::EPI && lane == 0) {
        info[0] = 0;
        for (int i = 0; i < C::NS; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], 1); }
        for (int i = 0; i < C::NB; ++i) { mbar_init(&t_full[i], 1); mbar_init(&t_empty[i], C::EPI); }
        mbar_init(done, 1);
        fence_mbarrier_init();
        prefetch_tensormap(&maps.a);
        prefetch_tensormap(&maps.w0);
        if (C::GU) prefetch_tensormap(&maps.w1);
    }
    if (warp == C::EPI + 1) {
        tmem_alloc(reinterpret_cast<uint32_t *>(info + 1), C::TMEM_COLS);
        tmem_relinquish();
        tc_fence_before();
    }
    const int KB = (p.K + kF8Block - 1) / kF8Block, nb = p.n_tiles;
    const int kb0 = KB * rank / split, nkb = KB * (rank + 1) / split - kb0;
    const int step = gridDim.x / split;
    Walk<C> wk;
    wk.start(blockIdx.x / split);
    bool have = !p.offsets && wk.get(p, cum);
    if (!p.offsets && warp == C::EPI && have && elect_one()) {
        // dense: the first weights are brought into L2 while the previous grid ends
        // (L2 is where that grid's writes arrive too, so nothing stale can be read)
        for (int i = 0; i < min(nkb, 2 * C::NS); ++i) {
            tma_prefetch_2d(&maps.w0, (kb0 + i) * kF8Block, wk.nt * 128);
            if (C::GU) tma_prefetch_2d(&maps.w1, (kb0 + i) * kF8Block, wk.nt * 128);
        }
    }
    if (p.offsets) {
        if (!p.early) grid_wait();
        build_groups<C>(p, cum, reinterpret_cast<int *>(tab));
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(info + 1);
    if (p.offsets) have = wk.get(p, cum);
    else if (!p.early) grid_wait();   // (the block is set up and its first tile known while the previous grid ends)
    // (once this block has its tensor memory: a block of the next grid on this SM
    // could otherwise take it and then wait for this grid; and after the wait, so
    // that an early reader of the next grid finds the grids before this complete)
    if (!p.early) grid_launch_dependents();
    RowTile tile{0, 0, 0, 0};   // the last tile whose sums are in `part` (split > 1: the only one)
    bool second = false;

    // the sums in `part` -> y or h: a warp per row, 4 columns a lane, the ranks' sums in rank order
    auto emit = [&](const RowTile &t) {
        const int n = t.nt * 128 + lane * 4;
        for (int j = rank + split * warp; j < t.rows; j += split * C::EPI) {
            float v[C::NW][4];
#pragma unroll
            for (int w = 0; w < C::NW; ++w) {
                const float *at = part + ((w * split * slice + (j * inverse >> 16)) * 128 + lane * 4);
                float4 s = *reinterpret_cast<const float4 *>(at);
                for (uint32_t r = 1; r < split; ++r) {
                    const float4 f = *reinterpret_cast<const float4 *>(at + r * slice * 128);
                    s.x += f.x; s.y += f.y; s.z += f.z; s.w += f.w;
                }
                v[w][0] = s.x; v[w][1] = s.y; v[w][2] = s.z; v[w][3] = s.w;
            }
            const int64_t row = t.row0 + j;
            if constexpr (C::GU) {
                float h[4], top = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[i] = n < p.N ? swiglu(v[0][i], v[1][i]) : 0.0f;   // (N is a multiple of 16)
                    top = fmaxf(top, finite_abs(h[i]));
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const int sp = f8_scale_exp(top);
                const float inv = pow2f(-sp);
                if (n < p.N)
                    *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(p.y) + row * p.N + n) =
                        f8x4_satfinite(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv);
                if (lane == 0) p.y_scale[row * nb + t.nt] = pow2f(sp);
            } else if (p.vec && n + 3 < p.N) {
                if (p.y_bf16) {
                    const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0][0], v[0][1]), hi = __floats2bfloat162_rn(v[0][2], v[0][3]);
                    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.y) + row * p.N + n) =
                        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
                } else {
                    *reinterpret_cast<float4 *>(static_cast<float *>(p.y) + row * p.N + n) =
                        make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < p.N) {
                        if (p.y_bf16) static_cast<__nv_bfloat16 *>(p.y)[row * p.N + n + i] = __float2bfloat16_rn(v[0][i]);
                        else static_cast<float *>(p.y)[row * p.N + n + i] = v[0][i];
                    }
            }
        }
    };

    if (warp == C::EPI) {
        // ---- TMA producer
        uint32_t it = 0;
        bool ok = true;
        auto load_w = [&](int s, int i) {
            uint8_t *st = smem + s * C::STAGE;
            mbar_arrive_expect_tx(&s_full[s], C::STAGE);
            tma_load_2d(st, &maps.w0, &s_full[s], (kb0 + i) * kF8Block, wk.e * p.N + wk.nt * 128);
            if (C::GU) tma_load_2d(st + C::W_BYTES, &maps.w1, &s_full[s], (kb0 + i) * kF8Block, wk.e * p.N + wk.nt * 128);
        };
        auto load_a = [&](int s, int i) {
            tma_load_2d(smem + s * C::STAGE + C::NW * C::W_BYTES, &maps.a, &s_full[s], (kb0 + i) * kF8Block, wk.row0);
        };
        bool waited = !p.early;
        for (; ok && have; wk.t += step, have = split == 1 && wk.get(p, cum)) {
            int i = 0;
            if (!waited && wk.e < p.E) {
                // the weights of the first stages are asked for before what the
                // previous kernel writes is waited for
                const int first = min(nkb, C::NS);
                if (lane == 0)
                    for (int j = 0; j < first; ++j) load_w(j, j);
                grid_wait();
                if (lane == 0)
                    for (int j = 0; j < first; ++j) load_a(j, j);
                waited = true;
                it = i = first;
            }
            for (; i < nkb && lane == 0 && wk.e < p.E; ++i, ++it) {
                const uint32_t s = it % C::NS;
                if (it >= C::NS && !bar_wait(&s_empty[s], ((it / C::NS) & 1) ^ 1, abort_flag, p.err)) { ok = false; break; }
                load_w(s, i);
                load_a(s, i);
            }
            ok = __shfl_sync(0xffffffffu, ok && !*abort_flag, 0);
        }
        if (lane == 0 && *abort_flag)   // wait for the copies in flight before the block leaves
            for (uint32_t j = it > C::NS ? it - C::NS : 0; j < it; ++j)
                mbar_wait(&s_full[j % C::NS], (j / C::NS) & 1, nullptr, p.err);
        __syncwarp();
    } else if (warp == C::EPI + 1) {
        // ---- MMA issuer
        constexpr uint32_t idesc = idesc_f8_f32(128, C::TN);
        if (p.early) grid_wait();   // (the wait for the previous grid is not one of the bounded ones)
        uint32_t it = 0;
        bool ok = true;
        for (; ok && have; wk.t += step, have = split == 1 && wk.get(p, cum)) {
            for (int i = 0; i < nkb && wk.e < p.E; ++i, ++it) {
                const uint32_t s = it % C::NS, b = it % C::NB;
                ok = bar_wait(&s_full[s], (it / C::NS) & 1, abort_flag, p.err) &&
                     (it < C::NB || bar_wait(&t_empty[b], ((it / C::NB) & 1) ^ 1, abort_flag, p.err));
                if (!__all_sync(0xffffffffu, ok)) break;
                tc_fence_after();
                const uint32_t st = smem_u32(smem) + s * C::STAGE;
                const uint64_t bd = smem_desc_k_sw128(st + C::NW * C::W_BYTES);
                if (elect_one()) {
#pragma unroll
                    for (int w = 0; w < C::NW; ++w) {
                        const uint64_t ad = smem_desc_k_sw128(st + w * C::W_BYTES);
#pragma unroll
                        for (int k = 0; k < 4; ++k)   // 32 bytes of K a step
                            tc_mma_f8(tmem + (b * C::NW + w) * C::TN, ad + 2 * k, bd + 2 * k, idesc, k != 0);
                    }
                    tc_commit(&t_full[b]);
                    tc_commit(&s_empty[s]);
                }
                __syncwarp();
            }
            ok = __all_sync(0xffffffffu, ok && !*abort_flag);
        }
        if (elect_one()) tc_commit(done);
        __syncwarp();
        if (lane == 0) mbar_wait(done, 0, nullptr, p.err);
        __syncwarp();
    } else {
        // ---- scale and sum: thread = one row of W
        if (p.early) grid_wait();
        const int w = warp >> 2, q = warp & 3, tid = threadIdx.x & 127;
        const uint32_t taddr = tmem + w * C::TN + ((uint32_t)(q * 32) << 16);
        float *mine = part + w * split * slice * 128 + tid;
        constexpr int PER = (C::SEG * C::TN + 127) / 128;
        float next[PER];
        // the scales' products of segment g of the tile at hand: [K block][row of a]
        auto fetch = [&](int g) {
            const float *sw = (w ? p.sw1 : p.sw0) + ((int64_t)wk.e * nb + wk.nt) * KB + kb0;
#pragma unroll
            for (int r = 0; r < PER; ++r) {
                const int v = r * 128 + tid, j = v / C::SEG, i = g * C::SEG + v % C::SEG;
                next[r] = v < C::SEG * C::TN && j < wk.rows && i < nkb && wk.e < p.E
                              ? __ldg(p.sa + (int64_t)(wk.row0 + j) * KB + kb0 + i) * __ldg(sw + i)
                              : 0.0f;
            }
        };
        uint32_t it = 0, half = 0;
        if (have) fetch(0);
        while (have) {
            float2 acc[C::TN / 2];
#pragma unroll
            for (int j = 0; j < C::TN / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);
            float *seg = tab;
            for (int i = 0; i < nkb && wk.e < p.E; ++i, ++it) {
                const int b = it % C::NB;
                if (i % C::SEG == 0) {
                    // (this half of the table was last read two segments ago, before
                    // the barrier of the one between)
                    seg = tab + half * C::TAB + w * C::SEG * C::TN;
                    half ^= 1;
#pragma unroll
                    for (int r = 0; r < PER; ++r) {
                        const int v = r * 128 + tid;
                        if (v < C::SEG * C::TN) seg[(v % C::SEG) * C::TN + v / C::SEG] = next[r];
                    }
                    named_barrier(1 + w, 128);
                    fetch(i / C::SEG + 1);
                }
                // (a thread that gives up still meets the others at the barriers)
                bar_wait(&t_full[b], (it / C::NB) & 1, abort_flag, p.err);
                __syncwarp();
                tc_fence_after();
                const float4 *s4 = reinterpret_cast<const float4 *>(seg + (i % C::SEG) * C::TN);
                const uint32_t from = taddr + b * C::NW * C::TN;
                constexpr int STEP = C::TN >= 32 ? 32 : 16;
#pragma unroll
                for (int c = 0; c < C::TN; c += STEP) {
                    uint32_t d[STEP];
                    if constexpr (STEP == 32) tmem_ld_32x32b_x32(from + c, d);
                    else tmem_ld_32x32b_x16(from + c, d);
                    tmem_ld_wait(d);
                    if (c + STEP == C::TN) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&t_empty[b]);
                    }
#pragma unroll
                    for (int j = 0; j < STEP; j += 4) {
                        const float4 s = s4[(c + j) / 4];
                        fma2(acc[(c + j) / 2], d[j], d[j + 1], s.x, s.y);
                        fma2(acc[(c + j) / 2 + 1], d[j + 2], d[j + 3], s.z, s.w);
                    }
                }
            }
            tile = {wk.e, wk.row0, wk.rows, wk.nt};
            wk.t += step;
            have = split == 1 && wk.get(p, cum);
            if (have) fetch(0);
            if (second) named_barrier(3, C::EPI * 32);       // the tile before has been written
            second = true;
            if (split == 1) {
#pragma unroll
                for (int j = 0; j < C::TN / 2; ++j) {
                    mine[2 * j * 128] = acc[j].x;
                    mine[(2 * j + 1) * 128] = acc[j].y;
                }
                named_barrier(3, C::EPI * 32);
                emit(tile);
            } else {
                // (no more tiles than clusters: each has one at most, and its walk ends there)
                cluster_wait();                              // every block of the cluster runs
                // this block's sums into its ring, which its products have left; then row j,
                // a warp per row, to rank j % split
                float *own = reinterpret_cast<float *>(smem) + w * C::TN * 128;
#pragma unroll
                for (int j = 0; j < C::TN / 2; ++j) {
                    own[2 * j * 128 + tid] = acc[j].x;
                    own[(2 * j + 1) * 128 + tid] = acc[j].y;
                }
                named_barrier(1 + w, 128);
                const uint32_t to = smem_u32(part + (w * split + rank) * slice * 128) + lane * 16;
                for (int j = q; j < tile.rows; j += 4) {
                    const uint32_t at = j * inverse >> 16;
                    st_cluster_f4(mapa_shared(to + at * 512, j - at * split), reinterpret_cast<const float4 *>(own + j * 128)[lane]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (split > 1) {
        if (warp >= C::EPI || !second) cluster_wait();       // (who has not met the first barrier above)
        cluster_sync_all();
        if (warp < C::EPI) emit(tile);
    }
    if (warp == C::EPI + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// Many rows: a on the MMA's M side, 128 rows a CTA (a CTA pair: 256, the W rows
// split between the two, which halves W's way through L2) times 256 rows of W
// (GU: 128 gate and 128 up rows, by 64 in turn, so that a thread holds a gate
// value and its up value).  In this orientation a thread's sums belong to one
// row of a and one block of W's rows, so its scale of a K block is one number.
// Persistent: every cluster takes tiles in turn; two accumulators in tensor
// memory let the MMAs of the next block (and of the next tile) run while one is
// taken out.  Bound by a K block's way from the MMA through the sums and back: 830
// clocks of a pair, 900 of a single CTA (whose 48 KB a K block also come near what
// an SM takes from L2), where the MMAs alone need 512.  2048 x 11008 x 4096 takes
// 79 us, 2.33 PFLOP/s, the tensor pipe busy for 55 % of the time.  Slower: four
// accumulators of N = 128 (107 us against 90 then), 16 summing warps of 64 sums
// (125 us against 108 then), tensor memory loads of 16 columns (86 us against 80).
//
// Roles: warps 0 .. 7 scale and sum (group w = warp / 4 takes columns 128 w ..
// 128 w + 127, 128 sums a thread), warp 8 loads by TMA, warp 9 issues the MMAs,
// warps 10 and 11 bring the scales to shared memory.
// ---------------------------------------------------------------------------
template <bool PAIR_, bool GU_>
struct LargeCfg {
    static constexpr bool PAIR = PAIR_, GU = GU_;
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int TM = 128 * CTAS;                    // rows of a
    static constexpr int TNW = GU ? 128 : 256;               // rows of W (of each, GU)
    static constexpr int W_ROWS = 256 / CTAS;                // W rows that a CTA holds
    static constexpr int W_BOX = GU ? 64 : 128;
    static constexpr int A_BYTES = 128 * 128;
    static constexpr int STAGE = A_BYTES + W_ROWS * 128;
    static constexpr int NS = GU ? (PAIR ? 6 : 4) : (PAIR ? 4 : 3);
    static constexpr int NB = 2;
    static constexpr int EPI = 8;
    static constexpr int THREADS = 384;                      // three warpgroups
    // registers a thread: 168 at launch (what 384 threads can have), then shifted
    // to the two summing warpgroups: 256 * 216 + 128 * 72 = 384 * 168
    static constexpr int REGS = 168, REGS_SUM = 216, REGS_REST = 72;
    static constexpr int GROUP = 8;                          // dense: row tiles that share a W tile in turn
    // scales: slots of SEG K blocks, [K block][128 rows of a, then 2 of W's blocks]
    static constexpr int SEG = 4, SLOTS = 4, SROW = 136;
    static constexpr int SLOT = SEG * SROW;                  // floats (a pitch of 136 spreads the K blocks over the banks)
    // a summing warp's 32 rows on their way out: boxes of 128 bytes a row (GU: one of
    // 64), swizzled as the store's tensor map has it
    static constexpr int OUT_BOX = GU ? 64 : 128;
    static constexpr int OUT_BYTES = GU ? 2048 : 8192;
    static constexpr int OFF_OUT = NS * STAGE;
    static constexpr int OFF_TOP = OFF_OUT + EPI * OUT_BYTES;     // GU: largest h of (tile parity, group, row)
    static constexpr int OFF_SC = OFF_TOP + (GU ? 2 * 2 * 128 * 4 : 0);
    static constexpr int OFF_BAR = OFF_SC + SLOTS * SLOT * 4;
    static constexpr int OFF_CUM = OFF_BAR + (2 * NS + 2 * NB + 2 * SLOTS + 1 + (GU ? 8 : 0)) * 8 + 24;   // (a multiple of 8)
    static constexpr int SMEM = OFF_CUM + 1024;              // + {row tiles before, first row} of each group of rows
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) large_kernel(const __grid_constant__ Maps maps, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float *tops = reinterpret_cast<float *>(smem + C::OFF_TOP);
    uint64_t *s_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *s_empty = s_full + C::NS, *t_full = s_empty + C::NS, *t_empty = t_full + C::NB;
    uint64_t *c_full = t_empty + C::NB, *c_empty = c_full + C::SLOTS, *done = c_empty + C::SLOTS;
    uint64_t *top_full = done + 1;                           // GU: of each tile parity and 32 rows
    int *info = reinterpret_cast<int *>(done + 1 + (C::GU ? 8 : 0));   // abort, TMEM base
    float *scales = reinterpret_cast<float *>(smem + C::OFF_SC);
    int2 *cum = reinterpret_cast<int2 *>(smem + C::OFF_CUM);
    volatile int *abort_flag = info;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = C::PAIR ? (int)cluster_ctarank() : 0;
    const int KB = (p.K + kF8Block - 1) / kF8Block;

    if (warp == C::EPI && lane == 0) {
        info[0] = 0;
        for (int i = 0; i < C::NS; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], 1); }
        for (int i = 0; i < C::NB; ++i) { mbar_init(&t_full[i], 1); mbar_init(&t_empty[i], C::EPI * C::CTAS); }
        for (int i = 0; i < C::SLOTS; ++i) { mbar_init(&c_full[i], 2); mbar_init(&c_empty[i], C::EPI); }
        mbar_init(done, 1);
        if (C::GU)
            for (int i = 0; i < 8; ++i) mbar_init(&top_full[i], 2);
        fence_mbarrier_init();
        prefetch_tensormap(&maps.a);
        prefetch_tensormap(&maps.w0);
        if (C::GU) prefetch_tensormap(&maps.w1);
    }
    if (warp == C::EPI + 1) {
        uint32_t *dst = reinterpret_cast<uint32_t *>(info + 1);
        if constexpr (C::PAIR) { tmem_alloc_pair(dst, 512); tmem_relinquish_pair(); }
        else { tmem_alloc(dst, 512); tmem_relinquish(); }
        tc_fence_before();
    }
    grid_wait();
    if (p.offsets) build_groups<C>(p, cum, reinterpret_cast<int *>(scales));
    __syncthreads();
    grid_launch_dependents();          // (this block has its tensor memory: see the small tiles)
    if (C::PAIR) cluster_sync_all();   // the peer's barriers are set up
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(info + 1);
    Walk<C> wk;
    wk.start(blockIdx.x / C::CTAS);
    if (warp >= C::EPI) reg_dealloc<C::REGS_REST>();

    if (warp == C::EPI) {
        // ---- TMA producer: this CTA's rows of a and share of W's rows
        const uint32_t full0 = C::PAIR ? mapa_shared(smem_u32(s_full), 0) : 0;
        uint32_t it = 0;
        bool ok = true;
        for (; ok && wk.get(p, cum); wk.t += gridDim.x / C::CTAS) {
            for (int i = 0; i < KB && lane == 0 && wk.e < p.E; ++i, ++it) {
                const uint32_t s = it % C::NS;
                if (it >= C::NS && !bar_wait(&s_empty[s], ((it / C::NS) & 1) ^ 1, abort_flag, p.err)) { ok = false; break; }
                uint8_t *st = smem + s * C::STAGE;
                if (rank == 0) mbar_arrive_expect_tx(&s_full[s], C::STAGE * C::CTAS);
                auto load = [&](uint8_t *dst, const CUtensorMap *m, int c1) {
                    if constexpr (C::PAIR) tma_load_2d_pair(dst, m, full0 + s * 8, i * kF8Block, c1);
                    else tma_load_2d(dst, m, &s_full[s], i * kF8Block, c1);
                };
                load(st, &maps.a, wk.row0 + 128 * rank);
                const int w_row = wk.e * p.N + wk.nt * C::TNW;
#pragma unroll
                for (int b = 0; b < C::W_ROWS / C::W_BOX; ++b) {
                    uint8_t *dst = st + C::A_BYTES + b * C::W_BOX * 128;
                    const int at = rank * (C::W_ROWS / C::W_BOX) + b;   // box of the whole W tile
                    if constexpr (C::GU) load(dst, at & 1 ? &maps.w1 : &maps.w0, w_row + (at >> 1) * C::W_BOX);
                    else load(dst, &maps.w0, w_row + at * C::W_BOX);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok && !*abort_flag, 0);
        }
        // (a launch that gave up: wait for the copies in flight before leaving)
        if (lane == 0 && *abort_flag && rank == 0)
            for (uint32_t j = it > C::NS ? it - C::NS : 0; j < it; ++j)
                mbar_wait(&s_full[j % C::NS], (j / C::NS) & 1, nullptr, p.err);
        __syncwarp();
    } else if (warp == C::EPI + 1) {
        // ---- MMA issuer (of a pair: its first CTA)
        constexpr uint32_t idesc = idesc_f8_f32(C::TM, 256);
        if (rank == 0) {
            uint32_t it = 0;
            bool ok = true;
            // (the whole warp walks and waits, one elected lane issues: in code that
            // only one thread runs, every MMA cost 115 clocks to issue)
            for (; ok && wk.get(p, cum); wk.t += gridDim.x / C::CTAS) {
                for (int i = 0; i < KB && wk.e < p.E; ++i, ++it) {
                    const uint32_t s = it % C::NS, b = it % C::NB;
                    ok = bar_wait(&s_full[s], (it / C::NS) & 1, abort_flag, p.err) &&
                         (it < C::NB || bar_wait(&t_empty[b], ((it / C::NB) & 1) ^ 1, abort_flag, p.err));
                    if (!__all_sync(0xffffffffu, ok)) break;
                    tc_fence_after();
                    const uint32_t st = smem_u32(smem) + s * C::STAGE;
                    const uint64_t ad = smem_desc_k_sw128(st), bd = smem_desc_k_sw128(st + C::A_BYTES);
                    const uint32_t dst = tmem + b * 256;
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {   // 32 bytes of K a step
                            if constexpr (C::PAIR) tc_mma_f8_pair(dst, ad + 2 * k, bd + 2 * k, idesc, k != 0);
                            else tc_mma_f8(dst, ad + 2 * k, bd + 2 * k, idesc, k != 0);
                        }
                        if constexpr (C::PAIR) { tc_commit_pair(&t_full[b]); tc_commit_pair(&s_empty[s]); }
                        else { tc_commit(&t_full[b]); tc_commit(&s_empty[s]); }
                    }
                    __syncwarp();
                }
                ok = __all_sync(0xffffffffu, ok && !*abort_flag);
            }
            if (elect_one()) {
                if constexpr (C::PAIR) tc_commit_pair(done);
                else tc_commit(done);
            }
            __syncwarp();
        }
    } else if (warp >= C::EPI + 2) {
        // ---- scales: this CTA's rows of a, and the tile's blocks of W (plain: two
        // blocks of rows; GU: gate and up), SEG K blocks at a time, 64 rows a warp
        const int half = (warp - C::EPI - 2) * 64;
        const int nb = (p.N + kF8Block - 1) / kF8Block;
        // of rows; a tile's first slot says which tile it is (the summing warps do not
        // walk themselves), and after the last tile one says so.
        uint32_t ck = 0;
        bool ok = true;
        for (bool more = true; ok && more; wk.t += gridDim.x / C::CTAS) {
            more = wk.get(p, cum);
            const int b0 = C::GU ? wk.nt : wk.nt * 2, b1 = C::GU ? b0 : min(b0 + 1, nb - 1);
            const int kbs = more && wk.e < p.E ? KB : 1;     // (tiles without a product: one slot, no scales)
            for (int i = 0; i < kbs; i += C::SEG, ++ck) {
                const uint32_t c = ck % C::SLOTS;
                ok = ck < C::SLOTS || bar_wait(&c_empty[c], ((ck / C::SLOTS) & 1) ^ 1, abort_flag, p.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                float *dst = scales + c * C::SLOT;
                if (i == 0 && half == 0 && lane == 0)
                    *reinterpret_cast<int4 *>(dst + 132) = make_int4(wk.e, wk.row0, more ? wk.rows : -1, wk.nt);
                if (more && wk.e < p.E) {
                    const int kb = min(i + (lane & 3), KB - 1);
                    const float *pa = p.sa + (int64_t)wk.row0 * KB + kb;
                    float f[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        f[r] = __ldg(pa + (int64_t)min(128 * rank + half + r * 8 + (lane >> 2), wk.rows - 1) * KB);
                    if (half == 0 && lane < 8) {
                        const float *pw = C::GU && (lane >> 2) ? p.sw1 : p.sw0;
                        dst[(lane & 3) * C::SROW + 128 + (lane >> 2)] =
                            __ldg(pw + ((int64_t)wk.e * nb + ((lane >> 2) ? b1 : b0)) * KB + kb);
                    }
#pragma unroll
                    for (int r = 0; r < 8; ++r) dst[(lane & 3) * C::SROW + half + r * 8 + (lane >> 2)] = f[r];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&c_full[c]);
            }
        }
    } else if (warp < C::EPI) {
        // ---- scale and sum: thread = one row of a, 128 columns
        reg_alloc<C::REGS_SUM>();
        const int w = warp >> 2, q = warp & 3, lrow = q * 32 + lane;
        const int nb = (p.N + kF8Block - 1) / kF8Block;
        const uint32_t taddr = tmem + w * 128 + ((uint32_t)(q * 32) << 16);
        const uint32_t empty0 = C::PAIR ? mapa_shared(smem_u32(t_empty), 0) : 0;
        uint8_t *out = smem + C::OFF_OUT + warp * C::OUT_BYTES;
        uint32_t it = 0, ck = 0;
        uint32_t turn = 0;                                   // tiles before this one
        for (;;) {
            // which tile
            if (!__all_sync(0xffffffffu, bar_wait(&c_full[ck % C::SLOTS], (ck / C::SLOTS) & 1, abort_flag, p.err))) break;
            const int4 tile = *reinterpret_cast<const int4 *>(scales + (ck % C::SLOTS) * C::SLOT + 132);   // e, row0, rows, nt
            __syncwarp();
            if (tile.z < 0) break;
            const int blocks = tile.x < p.E ? KB : 0;
            float2 acc[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) acc[j] = make_float2(0.0f, 0.0f);
            // The last 32 columns of a K block are summed while the first of the next
            // are on their way (d[1] and their scale go from one turn to the next).
            uint32_t d[2][32];
            float last = 0.0f;
#pragma unroll
            for (int j = 0; j < 32; ++j) d[1][j] = 0;
            if (blocks == 0) {
                if (lane == 0) mbar_arrive(&c_empty[ck % C::SLOTS]);
                ++ck;
            }
            for (int i = 0; i < blocks; ++i, ++it) {
                const uint32_t b = it % C::NB, c4 = ck % C::SLOTS, from = taddr + b * 256;
                if (i % C::SEG == 0) bar_wait(&c_full[c4], (ck / C::SLOTS) & 1, abort_flag, p.err);
                const float *sc = scales + c4 * C::SLOT + (i % C::SEG) * C::SROW;
                const float sa = sc[lrow], s0 = sa * sc[128 + (C::GU ? 0 : w)], s1 = C::GU ? sa * sc[129] : s0;
                bar_wait(&t_full[b], (it / C::NB) & 1, abort_flag, p.err);
                __syncwarp();
                tc_fence_after();
                tmem_ld_32x32b_x32(from, d[0]);
                if (i % C::SEG == C::SEG - 1 || i == blocks - 1) {
                    if (lane == 0) mbar_arrive(&c_empty[c4]);
                    ++ck;
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) fma2(acc[48 + j], d[1][2 * j], d[1][2 * j + 1], last);
#pragma unroll
                for (int c = 0; c < 3; ++c) {
                    tmem_ld_wait(d[c & 1]);
                    tmem_ld_32x32b_x32(from + 32 * (c + 1), d[(c + 1) & 1]);
#pragma unroll
                    for (int j = 0; j < 16; ++j) fma2(acc[c * 16 + j], d[c & 1][2 * j], d[c & 1][2 * j + 1], c < 2 ? s0 : s1);
                }
                last = s1;
                tmem_ld_wait(d[1]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (C::PAIR) mbar_arrive_cluster(empty0 + b * 8);
                    else mbar_arrive(&t_empty[b]);
                }
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) fma2(acc[48 + j], d[1][2 * j], d[1][2 * j + 1], last);
            const int wrow = 128 * rank + q * 32;            // this warp's first row of the tile
            const int left = tile.z - wrow;                  // and how many are the tile's
            const int64_t row = tile.y + wrow;
            const int nt = tile.w;
            // The rows leave by TMA, 32 rows of a box at a time: nothing waits for the
            // stores, which go out at 32 bytes a clock (64 KB a tile of bf16: 2000
            // clocks that overlap with the next tile).  A warp whose rows are not all
            // the tile's, and rows that are not 16-byte multiples, are written from
            // shared memory by the warp's lanes, a row's bytes by neighbouring lanes.
            auto at = [&](int box, int r, int chunk) {
                return out + box * 32 * C::OUT_BOX + r * C::OUT_BOX +
                       ((C::GU ? chunk ^ ((r >> 1) & 3) : chunk ^ (r & 7)) << 4);
            };
            auto emptied = [&] {   // the boxes sent before have been read
                if (lane == 0) bulk_wait_group_read<0>();
                __syncwarp();
            };
            // `boxes` boxes from column n0 on, elements of `elem` bytes
            auto send = [&](int boxes, int n0, auto elem_size, bool vec) {
                constexpr int elem = decltype(elem_size)::value, per = C::OUT_BOX / elem;   // columns of a box
                if (vec && left >= 32) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        for (int x = 0; x < boxes; ++x)
                            if (n0 + x * per < p.N) tma_store_2d(&maps.y, smem_u32(out) + x * 32 * C::OUT_BOX, n0 + x * per, (int)row);
                        bulk_commit_group();
                    }
                    return;
                }
                __syncwarp();
                uint8_t *y = static_cast<uint8_t *>(p.y) + row * p.N * elem;
                const int64_t pitch = (int64_t)p.N * elem;
                constexpr int CH = C::OUT_BOX / 16;          // chunks of a row
                for (int x = 0; x < boxes; ++x) {
                    const int col = n0 + x * per, bytes = min(per, p.N - col) * elem;
                    if (vec) {
                        for (int i = lane; i < 32 * CH; i += 32)
                            if (i / CH < left && i % CH * 16 < bytes)
                                *reinterpret_cast<uint4 *>(y + i / CH * pitch + (int64_t)col * elem + i % CH * 16) =
                                    *reinterpret_cast<const uint4 *>(at(x, i / CH, i % CH));
                    } else if constexpr (!C::GU) {
#pragma unroll
                        for (int l = 0; l < per / 32; ++l) {
                            const int b = (lane + 32 * l) * elem;
                            uint8_t *dst = y + (int64_t)col * elem + b;
#pragma unroll 8
                            for (int r = 0; r < 32; ++r) {
                                const uint8_t *src = at(x, r, b >> 4) + (b & 15);
                                if (r >= left || b >= bytes) continue;
                                if constexpr (elem == 2) *reinterpret_cast<uint16_t *>(dst + r * pitch) = *reinterpret_cast<const uint16_t *>(src);
                                else *reinterpret_cast<uint32_t *>(dst + r * pitch) = *reinterpret_cast<const uint32_t *>(src);
                            }
                        }
                    }
                }
                __syncwarp();
            };
            if constexpr (C::GU) {
                // h of features 64 w .. 64 w + 63 of the tile; the block's largest
                // over the two groups through shared memory
                const int n = nt * 128 + w * 64;
                float top = 0.0f;
                bool past = false;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    acc[j].x = swiglu(acc[j].x, acc[32 + j].x);
                    acc[j].y = swiglu(acc[j].y, acc[32 + j].y);
                    // (features past N: their W rows are zeros or another expert's)
                    if (j % 8 == 0 && n + 2 * j >= p.N) past = true;
                    if (past) acc[j] = make_float2(0.0f, 0.0f);
                    top = fmaxf(top, fmaxf(fabsf(acc[j].x), fabsf(acc[j].y)));   // (NaN is passed over)
                }
                if (top > 3.402823466e38f) {                 // an infinity: the largest finite value
                    top = 0.0f;
#pragma unroll
                    for (int j = 0; j < 32; ++j) top = fmaxf(top, fmaxf(finite_abs(acc[j].x), finite_abs(acc[j].y)));
                }
                float *t2 = tops + (turn & 1) * 2 * 128 + lrow;
                t2[w * 128] = top;
                // (a barrier in memory of the two warps of these rows, whose wait is
                // bounded: a warp that has given up does not come to this tile)
                uint64_t *both = &top_full[(turn & 1) * 4 + q];
                __syncwarp();
                if (lane == 0) mbar_arrive(both);
                bar_wait(both, (turn >> 1) & 1, abort_flag, p.err);
                top = fmaxf(t2[0], t2[128]);
                ++turn;
                const int sp = f8_scale_exp(top);
                const float inv = pow2f(-sp);
                emptied();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t u[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 lo = acc[c * 8 + 2 * k], hi = acc[c * 8 + 2 * k + 1];
                        u[k] = f8x4_satfinite(lo.x * inv, lo.y * inv, hi.x * inv, hi.y * inv);
                    }
                    *reinterpret_cast<uint4 *>(at(0, lane, c)) = make_uint4(u[0], u[1], u[2], u[3]);
                }
                // (N is a multiple of 16 and h 16-byte aligned)
                send(1, n, Bytes<1>{}, true);
                if (w == 0 && lane < left) p.y_scale[(row + lane) * nb + nt] = pow2f(sp);
            } else {
                const int n = nt * 256 + w * 128;
                if (p.y_bf16) {
                    emptied();
#pragma unroll
                    for (int c = 0; c < 16; ++c) {           // 8 columns
                        uint32_t u[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 f = acc[c * 4 + k];
                            const __nv_bfloat162 two = __floats2bfloat162_rn(f.x, f.y);
                            u[k] = *reinterpret_cast<const uint32_t *>(&two);
                        }
                        *reinterpret_cast<uint4 *>(at(c >> 3, lane, c & 7)) = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                    send(2, n, Bytes<2>{}, p.vec);
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {            // 64 columns
                        emptied();
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const float2 lo = acc[h * 32 + c * 2], hi = acc[h * 32 + c * 2 + 1];
                            *reinterpret_cast<float4 *>(at(c >> 3, lane, c & 7)) = make_float4(lo.x, lo.y, hi.x, hi.y);
                        }
                        send(2, n + h * 64, Bytes<4>{}, p.vec);
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_group_all();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    // (both CTAs of a pair: no commit's arrival is left on its way.  The wait is bounded,
    // so it begins when the sums have been taken out: the pair's second CTA issues
    // nothing, and from the kernel's start would wait as long as the product takes)
    if (warp == C::EPI + 1) {
        if (lane == 0) mbar_wait(done, 0, nullptr, p.err);
        __syncwarp();
    }
    // (of a pair: no CTA leaves while the other's MMAs may read its shared memory
    // or it may still arrive on the other's barriers)
    if (C::PAIR) cluster_sync_all();
    if (warp == C::EPI + 1) {
        tc_fence_after();
        if constexpr (C::PAIR) tmem_dealloc_pair(tmem, 512);
        else tmem_dealloc(tmem, 512);
    }
}

// ---- host -------------------------------------------------------------------

// Byte matrix [rows][K] in boxes of 128 columns, 128-byte swizzle, zeros past the edges.
static bool encode(CUtensorMap *m, const void *base, int64_t rows, int K, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)K};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static Params params(const Fp8Args &a) {
    Params p{};
    p.sa = a.a_scale;
    p.sw0 = a.w_scale;
    p.sw1 = a.w1_scale;
    p.offsets = a.offsets;
    p.y = a.y;
    p.y_scale = a.y_scale;
    p.err = a.err;
    p.M = a.M; p.N = a.N; p.K = a.K; p.E = a.E;
    p.y_bf16 = a.y_dtype == ZFFN_DT_BF16;
    return p;
}

// Row tiles of at most tr rows, at most: every expert may have one cut tile, and
// so may the rows of no expert.
static int64_t row_tiles_bound(const Fp8Args &a, int tr) {
    if (!a.offsets) return ((int64_t)a.M + tr - 1) / tr;
    return a.M / tr + (a.E + 1 < a.M ? a.E + 1 : a.M);
}

// Ask once a device for the largest share of shared memory, so that C::BLOCKS
// blocks run on an SM.
template <class C>
static cudaError_t prefer_shared() {
    static std::atomic<uint64_t> asked{0};
    const uint64_t bit = 1ull << (device_info().device & 63);
    if (asked.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(small_kernel<C>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess) asked.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Clusters of `split` small-tile blocks that the current device runs at once with
// one block an SM (asked once for each device and split, without the experts' table,
// so that the answer is not the first caller's: it counts one block an SM whatever
// the shared memory).
template <class C>
static int clusters_at_once(int split) {
    static std::atomic<int> known[64][C::MAX_SPLIT + 1];
    std::atomic<int> &k = known[device_info().device & 63][split];
    int n = k.load(std::memory_order_relaxed);
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(split);
        cfg.blockDim = dim3(C::THREADS);
        cfg.dynamicSmemBytes = C::SMEM;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = split;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, small_kernel<C>, &cfg) != cudaSuccess || n < 1) {
            cudaGetLastError();
            return 1;   // (no split for this call; the next one asks again)
        }
        k.store(n, std::memory_order_relaxed);
    }
    return n;
}

template <class C>
static cudaError_t launch_small(const Fp8Args &a, cudaStream_t s) {
    const DeviceInfo &di = device_info();
    Maps maps{};
    if (!encode(&maps.a, a.a, a.M, a.K, C::TN) || !encode(&maps.w0, a.w, (int64_t)a.E * a.N, a.K, 128) ||
        !encode(&maps.w1, C::GU ? a.w1 : a.w, (int64_t)a.E * a.N, a.K, 128))
        return cudaErrorInvalidValue;
    Params p = params(a);
    const int64_t rt = row_tiles_bound(a, C::TN), tiles = rt * f8_blocks(a.N), slots = (int64_t)di.num_sms * C::BLOCKS;
    const int KB = (int)f8_blocks(a.K);
    // fewer tiles than blocks: split K so that the blocks fill the SMs, two K blocks each at least
    const size_t smem = C::SMEM + (a.offsets ? ((size_t)a.E + 2) * 8 : 0);
    cudaError_t e = ensure_dynamic_smem((const void *)small_kernel<C>, smem);
    if (e == cudaSuccess) e = prefer_shared<C>();
    if (e != cudaSuccess) return e;
    int split = KB / 2 < C::MAX_SPLIT ? KB / 2 : C::MAX_SPLIT;
    if (split > slots / tiles) split = (int)(slots / tiles);
    // (all at once: a cluster's blocks lie within one part of the chip, so that fewer
    // of them run together than the SMs alone would take; a second wave costs more
    // than the split gains)
    while (split > 1 && (int64_t)clusters_at_once<C>(split) * C::BLOCKS < tiles) --split;
    if (split < 1) split = 1;
    const int64_t clusters = split > 1 || tiles < slots ? tiles : slots;
    if (tiles + slots > 0x7fffffff) return cudaErrorInvalidValue;
    p.row_tiles = (int)rt;
    p.n_tiles = (int)f8_blocks(a.N);
    p.early = a.early;
    p.vec = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.y) & (p.y_bf16 ? 7 : 15)) == 0;
    return launch_dependent(small_kernel<C>, dim3((unsigned)(clusters * split)), C::THREADS, smem, (unsigned)split, s, maps, p);
}

template <class C>
static cudaError_t launch_large(const Fp8Args &a, cudaStream_t s) {
    const DeviceInfo &di = device_info();
    Maps maps{};
    if (!encode(&maps.a, a.a, a.M, a.K, 128) || !encode(&maps.w0, a.w, (int64_t)a.E * a.N, a.K, C::W_BOX) ||
        !encode(&maps.w1, C::GU ? a.w1 : a.w, (int64_t)a.E * a.N, a.K, C::W_BOX))
        return cudaErrorInvalidValue;
    Params p = params(a);
    const int64_t rt = row_tiles_bound(a, C::TM), tiles = rt * ((a.N + C::TNW - 1) / C::TNW);
    if (tiles + di.num_sms > 0x7fffffff) return cudaErrorInvalidValue;
    p.row_tiles = (int)rt;
    p.n_tiles = (a.N + C::TNW - 1) / C::TNW;
    p.vec = a.N % (p.y_bf16 ? 8 : 4) == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
    int64_t clusters = di.num_sms / C::CTAS;
    if (tiles < clusters) clusters = tiles;
    if (C::GU || p.vec) {
        const int elem = C::GU ? 1 : p.y_bf16 ? 2 : 4;
        const cuuint64_t dims[2] = {(cuuint64_t)a.N, (cuuint64_t)a.M};
        const cuuint64_t strides[1] = {(cuuint64_t)a.N * elem};
        const cuuint32_t box[2] = {(cuuint32_t)(C::OUT_BOX / elem), 32};
        const cuuint32_t estr[2] = {1, 1};
        if (encode_fn()(&maps.y, elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                        2, a.y, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        C::GU ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    const size_t smem = C::SMEM + (a.offsets ? ((size_t)a.E + 2) * 8 : 0);
    // the registers' shift adds up only for the count that the kernel is launched with
    // (asked until it is known)
    static std::atomic<int> regs{0};
    if (regs.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes f{};
        const cudaError_t asked = cudaFuncGetAttributes(&f, large_kernel<C>);
        if (asked != cudaSuccess) return asked;
        regs.store(f.numRegs, std::memory_order_relaxed);
    }
    if (regs.load(std::memory_order_relaxed) != C::REGS) return cudaErrorInvalidConfiguration;
    const cudaError_t e = ensure_dynamic_smem((const void *)large_kernel<C>, smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(large_kernel<C>, dim3((unsigned)(clusters * C::CTAS)), C::THREADS, smem, C::CTAS, s, maps, p);
}

template <bool GU>
static cudaError_t launch(const Fp8Args &a, cudaStream_t s) {
    // rows a tile: the least of 16, 32, 64 that takes an expert's rows (with some
    // spread over their mean) at once, so that its weights are read once
    const int64_t mean = a.offsets ? ((int64_t)a.M * 3 / 2 + a.E - 1) / a.E : a.M;
    // many rows: the large tiles, where there are tiles for half of the SMs at least
    // (the small ones split K where there are fewer: 1856 rows of 2 experts times 136 x
    // 5136, 16 large tiles, 26 us; 240 blocks of small ones 12 us)
    const int64_t per = (a.N + LargeCfg<false, GU>::TNW - 1) / LargeCfg<false, GU>::TNW;
    const int64_t tiles = (a.M + 127) / 128 > a.E ? (a.M + 127) / 128 * per : (int64_t)a.E * per;
    // (whether the table of the experts' rows fits beside the tiles: gate/up up to 930 experts)
    const int room = device_info().max_smem_optin - (a.offsets ? (a.E + 2) * 8 : 0);
    if (LargeCfg<false, GU>::SMEM <= room && LargeCfg<true, GU>::SMEM <= room && a.M / a.E > 64 && tiles >= device_info().num_sms / 2) {
        // (pairs where few of their rows are past an expert's: 8 experts of 1024 rows
        // 211 -> 201 us, 128 of 256 rows 213 -> 242 us)
        if (a.M / a.E >= (a.offsets ? 1024 : 256)) return launch_large<LargeCfg<true, GU>>(a, s);
        return launch_large<LargeCfg<false, GU>>(a, s);
    }
    // (gate/up tiles of 32 rows have room for 622 experts' table, of 64 rows for 3954's)
    if (mean > 16 && mean <= 32 && SmallCfg<32, GU>::SMEM <= room) return launch_small<SmallCfg<32, GU>>(a, s);
    if (mean > 16 && SmallCfg<64, GU>::SMEM <= room) return launch_small<SmallCfg<64, GU>>(a, s);
    return launch_small<SmallCfg<16, GU>>(a, s);
}

}  // namespace f8

cudaError_t launch_fp8_matmul(const Fp8Args &a, cudaStream_t s) {
    if (!encode_fn()) return cudaErrorNotSupported;
    return a.w1 ? f8::launch<true>(a, s) : f8::launch<false>(a, s);
}

}  // namespace zffn
