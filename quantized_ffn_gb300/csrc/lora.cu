// lora.cu -- low-rank adapters of many requests at once.  With the tokens sorted by
// adapter (rows), e the adapter of a row and t its token:
//     shrink   v[row]  = scale[e] x[t] W_e^T      fp32 [T][r]
//     expand   out[t]  = base[t] + v[row] W_e^T
//     outer    d_e     = sum over e's rows of v[row]^T x[t]
// The forward pass is shrink by A and expand by B; the way back shrink of dy by B,
// expand by A, and two outer products.  r is small (8 to 128), so each is bound by the
// tokens' rows, which are gathered (and written back) by their tokens where they lie.
//
// Tensor cores take bf16, and v is fp32: it goes as the sum of three bf16 pieces of 8
// bits each, which is exact, so that v is not rounded between the products.  Shrink writes
// them beside v, [T][3 up16(r), to the next 64], so that expand and outer load them by TMA: split in the
// blocks that multiply them, once for each tile of columns, they were outer's bound (4096
// rows of r = 32: 62 us for both outer products).
#include <atomic>

#include <algorithm>
#include <type_traits>

#include "bf16.h"
#include "groups.cuh"
#include "launch.cuh"
#include "roles.cuh"
#include "tiles.cuh"

namespace zffn {
namespace lora {

// ---- pieces -----------------------------------------------------------------

// 16 bytes global -> shared, or 16 zero bytes (the address is then not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool some) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(some ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// Shared memory to another rank's, completion counted on a barrier there.
__device__ __forceinline__ void copy_to_rank(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "r"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ float lo_f32(uint32_t two) { return __uint_as_float(two << 16); }
__device__ __forceinline__ float hi_f32(uint32_t two) { return __uint_as_float(two & 0xFFFF0000u); }
// v = p[0] + p[1] + p[2], bf16 values in the high halves: v's bits cut after 8 and 16
// (differences of values that agree so far are exact).  Infinities and NaN stay in p[0].
__device__ __forceinline__ void pieces(float v, uint32_t (&p)[3]) {
    p[0] = __float_as_uint(v) & 0xFFFF0000u;
    const float rest = v - __uint_as_float(p[0]);
    p[1] = __float_as_uint(rest) & 0xFFFF0000u;
    p[2] = __float_as_uint(rest - __uint_as_float(p[1]));
    if (!(fabsf(v) <= 3.402823466e38f)) {
        p[0] = v != v ? 0x7FFF0000u : p[0];
        p[1] = p[2] = 0;
    }
}
__device__ __forceinline__ uint32_t high_halves(uint32_t lo, uint32_t hi) { return __byte_perm(lo, hi, 0x7632); }
// A quad of v's row to its three places.
__device__ __forceinline__ void put_pieces(__nv_bfloat16 *row, int r16, int c, float4 f) {
    uint32_t a[4][3];
    pieces(f.x, a[0]); pieces(f.y, a[1]); pieces(f.z, a[2]); pieces(f.w, a[3]);
#pragma unroll
    for (int k = 0; k < 3; ++k)
        *reinterpret_cast<uint2 *>(row + k * r16 + c) = make_uint2(high_halves(a[0][k], a[1][k]), high_halves(a[2][k], a[3][k]));
}
__host__ __device__ constexpr int up16(int r) { return (r + 15) / 16 * 16; }
// Values of a row of pieces: whole boxes of 64, so that one copy takes them all (what is past
// the third piece is neither written nor used).
__host__ __device__ constexpr int pieces_pitch(int r) { return (3 * up16(r) + 63) / 64 * 64; }

struct Params {
    const int32_t *row_slot, *slot_row, *offsets;
    const float *scale;
    int *err;
    int T, r, L, C;
    FastDiv each, by_quads, by_wide;   // of the walk; by the float4s of a row of v, up to 16 values; by its pieces' 16 bytes
};

// ---------------------------------------------------------------------------
// Shrink on the tensor cores: 128 rows (on the MMA's M side) times all r rows of W.  The
// blocks of a cluster share the contraction; rows 128 / split * i and on are added up by
// rank i, in rank order.  The tensor core's adds drop what is below the accumulator's last
// bit (positive values: of 512 2.3e-7 short, of 2048 2.3e-6, of 32768 1.5e-4): S_PART stages, 512 values,
// go to an accumulator, then the next, of two or four, whose sums meet in registers.  A block
// with more stages than that takes turns: when all accumulators are full their sum goes to the
// first one, and the others begin again (2.4e-7 short whatever the length).
// A tile whose tokens follow one another (a packed sequence) is loaded by TMA, another
// gathered by 16-byte copies.  (The copy engine's own gather takes four rows of 128 bytes at a
// time, and about 100 clocks for it.)  A stage takes 0.3 to 0.5 us whatever the number of
// stages: 2048 rows of 4096 values, 8 adapters, r = 64, 16 us (8 stages a block and their join),
// 4096 rows of 11008, r = 32, 24 us, 3.8 TB/s; a cluster of four took 20.5 -> 25 us at 16 tokens.
//
// Roles: warps 0 .. 3 gather x's rows, then take the sums out; warp 4 loads W, and x's
// rows where they follow one another, warp 5 issues the MMAs.
// ---------------------------------------------------------------------------
constexpr int S_NS = 4, S_LAG = 3, S_THREADS = 192, S_MAX_SPLIT = 8, S_PART = 8;

// W's bytes of a stage: K-major [r][64], or MN-major boxes [64][64]
__host__ __device__ constexpr int s_w_bytes(int r, bool mn) { return mn ? (r + 63) / 64 * 8192 : up16(r) * 128; }
static size_t s_smem(int r, bool mn) { return 1024 + (size_t)S_NS * (16384 + s_w_bytes(r, mn)) + (2 * S_NS + 3) * 8 + 8; }

template <bool MN>
__global__ void __launch_bounds__(S_THREADS) shrink_kernel(const __grid_constant__ CUtensorMap xm, const __grid_constant__ CUtensorMap w, const Params p,
                                                           const __nv_bfloat16 *x, float *v, __nv_bfloat16 *v16,
                                                           const float *other, __nv_bfloat16 *other16) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint32_t split;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(split));
    const uint32_t rank = cluster_ctarank();
    const int wb = s_w_bytes(p.r, MN), stage = 16384 + wb;
    // once the stages are idle: sums [rank][row / split][r] from every rank, and this one's own
    float *part = reinterpret_cast<float *>(smem), *own = part + 128 * p.r;
    uint64_t *s_full = reinterpret_cast<uint64_t *>(smem + S_NS * stage);
    uint64_t *s_empty = s_full + S_NS, *t_full = s_empty + S_NS, *t_empty = t_full + 1, *j_full = t_full + 2;
    int *info = reinterpret_cast<int *>(j_full + 1);         // abort, TMEM base
    volatile int *abort_flag = info;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    const int r16 = up16(p.r), cols = r16 <= 32 ? 32 : r16 <= 64 ? 64 : 128, accs = cols <= 64 ? 4 : 2;
    if (tid == 0) {
        info[0] = 0;
        for (int i = 0; i < S_NS; ++i) { mbar_init(&s_full[i], 5); mbar_init(&s_empty[i], 1); }
        mbar_init(t_full, 1);
        mbar_init(t_empty, 4);
        mbar_init(j_full, 1);
        mbar_arrive_expect_tx(j_full, 128 * p.r * 4);
        fence_mbarrier_init();
    }
    if (warp == 4 && lane == 0) {
        prefetch_tensormap(&xm);
        prefetch_tensormap(&w);
    }
    if (warp == 5) {
        tmem_alloc(reinterpret_cast<uint32_t *>(info + 1), cols * accs);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    grid_wait();
    grid_launch_dependents();          // (this block has its tensor memory)
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(info + 1);
    GroupWalk<128, 1> wk;
    wk.start(p.offsets, p.T, p.L, 1, p.each, true, blockIdx.x / split);
    const bool have = wk.get(), some = have && wk.e < p.L;
    const int blocks = (p.C + KB - 1) / KB;
    // this rank's stages: every split-th, so that the ranks read neighbouring columns at a time
    const int nkb = (blocks - (int)rank + (int)split - 1) / (int)split;
    auto block_of = [&](int i) { return i * (int)split + (int)rank; };
    // stages of the first turn, of each after it (the first accumulator holds the sum so far); turns
    // before the last, and the last one's parts besides the first accumulator
    const int first_turn = accs * S_PART, turn = first_turn - S_PART;
    const int turns = nkb > first_turn ? (nkb - first_turn + turn - 1) / turn : 0;
    const int more = turns ? (nkb - first_turn - (turns - 1) * turn + S_PART - 1) / S_PART : (nkb + S_PART - 1) / S_PART - 1;
    const float scale = some && p.scale ? __ldcg(p.scale + wk.e) : 1.0f;

    // the tile's tokens, 4 lane + j, and whether they follow one another
    int tok[4];
    bool packed = true;
    if (some && warp < 5) {
#pragma unroll
        for (int j = 0; j < 4; ++j) tok[j] = lane * 4 + j < wk.rows ? __ldcg(p.row_slot + wk.row0 + lane * 4 + j) : -1;
        const int t0 = __shfl_sync(0xffffffffu, tok[0], 0);
        packed = t0 >= 0 && t0 <= p.T - wk.rows;             // (any word may be there: no sum of it before that)
        for (int j = 0; j < 4; ++j) packed = packed && (lane * 4 + j >= wk.rows || tok[j] == t0 + lane * 4 + j);
        packed = __all_sync(0xffffffffu, packed);
    }

    // 16 columns of this warp's rows, summed over the first accumulator and n others
    auto sum_of = [&](int c, int n, uint32_t (&d)[16]) {
        const uint32_t at = tmem + ((uint32_t)(warp * 32) << 16) + c;
        tmem_ld_32x32b_x16(at, d);
        tmem_ld_wait(d);
        for (int k = 1; k <= n; ++k) {
            uint32_t other_d[16];
            tmem_ld_32x32b_x16(at + k * cols, other_d);
            tmem_ld_wait(other_d);
#pragma unroll
            for (int j = 0; j < 16; ++j) d[j] = __float_as_uint(__uint_as_float(d[j]) + __uint_as_float(other_d[j]));
        }
    };
    if (some && warp < 4) {
        // ---- gather: thread = one 16-byte column of rows tid / 8 + 16 i
        int joined = 0;                // turns whose sums have gone to the first accumulator
        auto join = [&] {
            const bool ok = bar_wait_warp(t_full, joined & 1, abort_flag, p.err);
            if (!ok) return false;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < p.r; c += 16) {
                uint32_t d[16];
                sum_of(c, accs - 1, d);
                tmem_st_32x32b_x16(tmem + ((uint32_t)(warp * 32) << 16) + c, d);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(t_empty);
            ++joined;
            return true;
        };
        if (!packed) {
            const int chunk = tid & 7, first = tid >> 3;
            const uint32_t dst = smem_u32(smem) + first * 128 + ((chunk ^ (first & 7)) << 4);
            const __nv_bfloat16 *src[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int row = first + 16 * i, t = row < wk.rows ? __ldcg(p.row_slot + wk.row0 + row) : -1;
                src[i] = (unsigned)t < (unsigned)p.T ? x + (int64_t)t * p.C + chunk * 8 : nullptr;
            }
            bool ok = true;
            auto filled = [&](int i) {     // this thread's copies of stage i have arrived
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_full[i % S_NS]);
            };
            for (int i = 0; i < nkb; ++i) {
                const int s = i % S_NS, c = block_of(i) * KB;
                if (i >= S_NS) ok = bar_wait_warp(&s_empty[s], ((i / S_NS) & 1) ^ 1, abort_flag, p.err);
                if (!ok) break;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool there = src[j] && c + chunk * 8 < p.C;
                    copy16(dst + s * stage + j * 2048, there ? src[j] + c : x, there);
                }
                copy_commit();
                if (i >= S_LAG) {
                    copy_wait<S_LAG>();
                    filled(i - S_LAG);
                    // (a turn's last stage: the stages begun since wait for no later one)
                    if (joined < turns && i - S_LAG == first_turn + joined * turn - 1) ok = join();
                    if (!ok) break;
                }
            }
            copy_wait<0>();
            if (ok)
                for (int i = nkb > S_LAG ? nkb - S_LAG : 0; i < nkb; ++i) filled(i);
        }
        while (joined < turns && join()) {}
    } else if (some && warp == 4) {
        // ---- by TMA: W, and a packed tile's rows (past the adapter's last: rows that nothing takes)
        const int t0 = __shfl_sync(0xffffffffu, tok[0], 0);
        int i = 0;
        for (bool ok = true; i < nkb; ++i) {
            const int s = i % S_NS;
            if (i >= S_NS) ok = bar_wait_warp(&s_empty[s], ((i / S_NS) & 1) ^ 1, abort_flag, p.err);
            if (!ok) break;
            uint8_t *to = smem + s * stage;
            if (lane == 0) {
                mbar_arrive_expect_tx(&s_full[s], (packed ? 16384 : 0) + (MN ? wb : p.r * 128));
                if (packed) tma_load_2d(to, &xm, &s_full[s], block_of(i) * KB, t0);
                if constexpr (MN) {
                    for (int b = 0; b * 64 < p.r; ++b) tma_load_3d(to + 16384 + b * 8192, &w, &s_full[s], b * 64, block_of(i) * KB, wk.e);
                } else {
                    tma_load_3d(to + 16384, &w, &s_full[s], block_of(i) * KB, 0, wk.e);
                }
            } else if (packed && lane < 5) {
                mbar_arrive(&s_full[s]);   // (for the gathering warps)
            }
            __syncwarp();
        }
        if (lane == 0 && *abort_flag)  // wait for the copies in flight before the block leaves
            for (int j = i > S_NS ? i - S_NS : 0; j < i; ++j) mbar_wait(&s_full[j % S_NS], (j / S_NS) & 1, nullptr, p.err);
        __syncwarp();
    } else if (some && warp == 5) {
        // ---- MMA issuer
        const uint32_t idesc = idesc_bf16_f32(128, r16, false, MN);
        bool ok = true;
        uint32_t dst = tmem;
        int turned = 0, full = 0;      // turns joined; commits on t_full
        for (int i = 0, at = 0; i < nkb; ++i, ++at) {
            const int s = i % S_NS;
            if (at == S_PART) at = 0, dst += cols;
            if (at == 0 && dst == tmem + accs * cols) {      // (the last turn's sums have been joined)
                ok = bar_wait_warp(t_empty, turned & 1, abort_flag, p.err);
                if (!ok) break;
                ++turned;
                dst = tmem + cols;
            }
            const bool last = i == nkb - 1 || (at == S_PART - 1 && dst == tmem + (accs - 1) * cols);
            ok = bar_wait_warp(&s_full[s], (i / S_NS) & 1, abort_flag, p.err);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sx = smem_u32(smem) + s * stage;
            const int n = (min(KB, p.C - block_of(i) * KB) + 15) / 16;
            const uint64_t xd = smem_desc_k_sw128(sx), wd = MN ? smem_desc_mn_sw128(sx + 16384, 8192) : smem_desc_k_sw128(sx + 16384);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < KB / 16; ++k) {
                    if (k >= n) break;
                    tc_mma_bf16(dst, xd + k * k_step(false), wd + k * k_step(MN), idesc, (at | k) != 0);
                }
                tc_commit(&s_empty[s]);
                if (last) tc_commit(t_full);
            }
            __syncwarp();
            full += last;
        }
        if (!ok) {                     // (nothing issued is left on its way)
            if (elect_one()) tc_commit(t_full);
            __syncwarp();
            if (lane == 0) mbar_wait(t_full, full & 1, nullptr, p.err);
            __syncwarp();
        }
    }
    if (have && warp < 4) {
        // ---- take out: thread = one row
        if (some) {
            bar_wait_warp(t_full, turns & 1, abort_flag, p.err);
            tc_fence_after();
        }
        const int row = tid;
        float *to = v + (int64_t)(wk.row0 + row) * p.r;
        __nv_bfloat16 *to16 = v16 + (int64_t)(wk.row0 + row) * pieces_pitch(p.r);
        const bool join = some && split > 1;
        if (join) cluster_sync_all();                        // every block's stages are idle
        for (int c = 0; c < p.r; c += 16) {
            uint32_t d[16];
            if (some) {
                sum_of(c, more, d);
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) d[j] = 0;
            }
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                float4 f = make_float4(__uint_as_float(d[j]), __uint_as_float(d[j + 1]), __uint_as_float(d[j + 2]), __uint_as_float(d[j + 3]));
                if (join) {
                    if (c + j < p.r) *reinterpret_cast<float4 *>(own + row * p.r + c + j) = f;
                    continue;
                }
                if (row >= wk.rows) continue;
                f.x *= scale; f.y *= scale; f.z *= scale; f.w *= scale;
                if (c + j < p.r) *reinterpret_cast<float4 *>(to + c + j) = f;
                else f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (some) put_pieces(to16, r16, c + j, f);
            }
        }
        if (join) {
            // rows 128 / split * i and on to rank i (written by the lanes, 16 bytes each, they
            // took 8000 clocks for r = 64)
            fence_proxy_async_smem();
            named_barrier(1, 128);
            if (tid < (int)split) {
                const uint32_t bytes = 128 / split * p.r * 4;
                copy_to_rank(mapa_shared(smem_u32(part) + rank * bytes, tid), smem_u32(own) + tid * bytes, bytes, mapa_shared(smem_u32(j_full), tid));
            }
        }
        tc_fence_before();
    } else if (some && split > 1) {
        cluster_sync_all();
    }
    __syncthreads();
    if (some && split > 1) {
        volatile int never = 0;        // (the rows come also from a rank that gave up)
        bar_wait_warp(j_full, 0, &never, p.err);
        const int per = 128 / split, quads = r16 / 4;
        for (int i = tid; i < per * quads; i += S_THREADS) {
            const int lrow = p.by_quads.div(i), row = rank * per + lrow, c = (i - lrow * quads) * 4;
            if (row >= wk.rows) break;
            float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (c < p.r) {
                f = *reinterpret_cast<const float4 *>(part + lrow * p.r + c);
                for (uint32_t k = 1; k < split; ++k) {
                    const float4 g = *reinterpret_cast<const float4 *>(part + (k * per + lrow) * p.r + c);
                    f.x += g.x; f.y += g.y; f.z += g.z; f.w += g.w;
                }
                f.x *= scale; f.y *= scale; f.z *= scale; f.w *= scale;
                *reinterpret_cast<float4 *>(v + (int64_t)(wk.row0 + row) * p.r + c) = f;
            }
            put_pieces(v16 + (int64_t)(wk.row0 + row) * pieces_pitch(p.r), r16, c, f);
        }
    }
    if (some && other) {
        // the other outer product's rows of this tile
        const int per = 128 / split, quads = r16 / 4;
        for (int i = tid; i < per * quads; i += S_THREADS) {
            const int lrow = p.by_quads.div(i), row = rank * per + lrow, c = (i - lrow * quads) * 4;
            if (row >= wk.rows) break;
            const float4 f = c < p.r ? __ldcg(reinterpret_cast<const float4 *>(other + (int64_t)(wk.row0 + row) * p.r + c)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            put_pieces(other16 + (int64_t)(wk.row0 + row) * pieces_pitch(p.r), r16, c, f);
        }
    }
    if (some && split > 1) cluster_sync_all();               // (no block leaves while its rows are on their way)
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, cols * accs);
    }
}

// ---------------------------------------------------------------------------
// Expand on the tensor cores: 128 sorted rows times TN columns of out.  A block keeps one
// row tile's pieces of v and takes every G-th tile of the columns.  base's rows come to
// shared memory as boxes of 32 rows x 128 bytes, NB tiles of them in turn, the sums are added
// there and the boxes leave: by TMA where the tile's tokens follow one another, else by
// 16-byte copies and stores.  (Loads to registers pass through L1, which is 28 KB beside this
// kernel's shared memory: no more than that was on its way, and 2048 x 11008 took 38 us.  Now
// 26 us, 3.5 TB/s: bound by a tile's way from base through the sums and out.)  base and W are
// asked for before the grid that writes v has ended.
//
// Roles: warps 0 .. 7 take 32 rows and half of the columns each, with boxes of their own;
// warp 8 loads v and W and issues the MMAs, warps 9 .. 11 copy base to out for tokens of no
// adapter.
// ---------------------------------------------------------------------------
constexpr int E_WARPS = 8, E_THREADS = (E_WARPS + 4) * 32;

template <int ELEM_, int TN_, int BOXES_, bool MN_>
struct ExpandCfg {
    static constexpr int ELEM = ELEM_, TN = TN_, BOXES = BOXES_;   // BOXES: 64-wide boxes of r
    static constexpr bool MN = MN_;
    static constexpr int V_BYTES = 3 * BOXES * 16384;        // the pieces
    static constexpr int W_BYTES = BOXES * TN * 128;         // of a tile; two in turn
    static constexpr int PER = 128 / ELEM;                   // columns of a box
    static constexpr int OWN = TN / 2 / PER;                 // boxes of a warp and tile
    static constexpr int TILE = 128 * TN * ELEM;
    static constexpr int ROOM = (224 * 1024 - V_BYTES - 2 * W_BYTES) / TILE, NB = ROOM > 4 ? 4 : ROOM;
    static_assert(NB >= 2, "one tile comes while another leaves");
    static constexpr int AHEAD = NB > 2 ? NB - 2 : 1;        // tiles that base is asked for ahead; the others' leave
    static constexpr int OFF_W = V_BYTES;
    static constexpr int OFF_BOX = OFF_W + 2 * W_BYTES;
    static constexpr int OFF_BAR = OFF_BOX + NB * TILE;
    static constexpr int SMEM = 1024 + OFF_BAR + (9 + E_WARPS * NB) * 8 + 8;
    static constexpr int TMEM_COLS = 2 * TN;
};

template <class C>
__global__ void __launch_bounds__(E_THREADS, 1) expand_kernel(const __grid_constant__ CUtensorMap vm, const __grid_constant__ CUtensorMap w,
                                                              const __grid_constant__ CUtensorMap bm, const __grid_constant__ CUtensorMap om,
                                                              const Params p, const void *base, void *out, int sms, int G) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *w_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *w_empty = w_full + 2, *t_full = w_full + 4, *t_empty = w_full + 6, *v_full = w_full + 8, *b_full = w_full + 9;
    int *info = reinterpret_cast<int *>(b_full + E_WARPS * C::NB);   // abort, TMEM base
    volatile int *abort_flag = info;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    const int r16 = up16(p.r);
    if (tid == 0) {
        info[0] = 0;
        mbar_init(v_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&w_full[i], 1);
            mbar_init(&w_empty[i], 1);
            mbar_init(&t_full[i], 1);
            mbar_init(&t_empty[i], E_WARPS);
        }
        for (int i = 0; i < E_WARPS * C::NB; ++i) mbar_init(&b_full[i], 1);
        fence_mbarrier_init();
    }
    if (warp == E_WARPS && lane == 0) {
        prefetch_tensormap(&vm);
        prefetch_tensormap(&w);
        prefetch_tensormap(&om);
        if (base) prefetch_tensormap(&bm);
    }
    if (warp == E_WARPS) {
        tmem_alloc(reinterpret_cast<uint32_t *>(info + 1), C::TMEM_COLS);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(info + 1);
    // (what the grid before this one does not write may be read before its end: it let this
    // one start after the grids before it had ended)
    GroupWalk<128, 1> wk;
    wk.start(p.offsets, p.T, p.L, 1, p.each, false, 0);
    // (G blocks to a row tile, as many as run at once: of the tiles that there are, else, past 128
    // groups, whose counting would take microseconds, of those that there may be; 2048 tokens of
    // 64 adapters, r = 16: 151 us by those that there may be)
    if (p.L <= 128) {
        int tiles = __shfl_sync(0xffffffffu, wk.inc, 31);
        while (wk.e0 + 32 <= p.L) {
            wk.hold(wk.e0 + 32);
            tiles += __shfl_sync(0xffffffffu, wk.inc, 31);
        }
        if (wk.e0) wk.start(p.offsets, p.T, p.L, 1, p.each, false, 0);
        G = max(1, sms / max(1, tiles));
    }
    wk.t = blockIdx.x / G;
    const bool have = wk.get();
    const int n_tiles = (p.C + C::TN - 1) / C::TN, g = blockIdx.x % G;
    const bool any = have && g < n_tiles;
    const int64_t pitch = (int64_t)p.C * C::ELEM;

    // warps 0 .. 7: lane i holds the token of its i-th row, -1 for none
    const int quarter = warp & 3, half = warp >> 2, left = wk.rows - quarter * 32;
    const bool mine = any && warp < E_WARPS && left > 0;
    int token = -1;
    bool packed = false;
    if (mine) {
        if (lane < left) token = __ldcg(p.row_slot + wk.row0 + quarter * 32 + lane);
        if ((unsigned)token >= (unsigned)p.T) token = -1;
        const int t0 = __shfl_sync(0xffffffffu, token, 0);
        packed = __all_sync(0xffffffffu, lane >= left || token == t0 + lane) && t0 >= 0;
    }
    auto box = [&](int b, int x) { return smem + C::OFF_BOX + b * C::TILE + (warp * C::OWN + x) * 4096; };
    auto column = [&](int nt, int x) { return nt * C::TN + half * (C::TN / 2) + x * C::PER; };
    auto place = [&](const void *of, int t, int col, int chunk) {
        return reinterpret_cast<uint4 *>(static_cast<uint8_t *>(const_cast<void *>(of)) + t * pitch + (int64_t)col * C::ELEM + chunk * 16);
    };
    auto chunks = [&](int col) { return min(8, (p.C - col) * C::ELEM / 16); };   // 16-byte columns of a box that are out's
    auto ask = [&](int nt, int b) {    // base's part of tile nt into buffers b
        if (!base) return;
        if (packed) {
            if (lane == 0) {
                uint64_t *bar = &b_full[warp * C::NB + b];
                mbar_arrive_expect_tx(bar, C::OWN * 4096);
                for (int x = 0; x < C::OWN; ++x) tma_load_2d(box(b, x), &bm, bar, column(nt, x), token);
            }
            __syncwarp();
            return;
        }
        for (int x = 0; x < C::OWN; ++x) {
            const int col = column(nt, x), n = chunks(col);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = i * 4 + (lane >> 3), t = __shfl_sync(0xffffffffu, token, r);
                if (t >= 0 && (lane & 7) < n)
                    copy16(smem_u32(box(b, x)) + r * 128 + (((lane & 7) ^ (r & 7)) << 4), place(base, t, col, lane & 7), true);
            }
        }
    };
    auto load_w = [&](int nt, int b) {
        uint8_t *to = smem + C::OFF_W + b * C::W_BYTES;
        if constexpr (C::MN) {
            mbar_arrive_expect_tx(&w_full[b], C::TN / 64 * r16 * 128);
            for (int x = 0; x < C::TN / 64; ++x) tma_load_3d(to + x * r16 * 128, &w, &w_full[b], nt * C::TN + x * 64, 0, wk.e);
        } else {
            const int boxes = (p.r + 63) / 64;
            mbar_arrive_expect_tx(&w_full[b], boxes * C::TN * 128);
            for (int x = 0; x < boxes; ++x) tma_load_3d(to + x * C::TN * 128, &w, &w_full[b], x * 64, nt * C::TN, wk.e);
        }
    };
    if (mine) {
        for (int i = 0; i < C::AHEAD; ++i) {
            if (g + i * G < n_tiles) ask(g + i * G, i);
            copy_commit();
        }
    } else if (any && warp == E_WARPS && lane == 0) {
        load_w(g, 0);
        if (g + G < n_tiles) load_w(g + G, 1);
    }
    grid_wait();
    grid_launch_dependents();

    if (any && warp < E_WARPS) {
        int i = 0, b = 0;
        uint32_t phases = 0;
        bool ok = true;
        for (int nt = g; nt < n_tiles; nt += G, ++i) {
            const int acc = i & 1;
            if (mine) {
                // the tile before (NB > 2: the one before that) has left its buffers: the base
                // AHEAD tiles on goes there
                const int next = nt + C::AHEAD * G;
                if (lane == 0) bulk_wait_group_read<(C::NB > 2 ? 1 : 0)>();
                __syncwarp();
                if (next < n_tiles) ask(next, (b + C::AHEAD) % C::NB);
                copy_commit();
            }
            ok = bar_wait_warp(&t_full[acc], (i >> 1) & 1, abort_flag, p.err);
            if (mine && base) {
                if (packed) ok = ok && bar_wait_warp(&b_full[warp * C::NB + b], (phases >> b) & 1, abort_flag, p.err);
                else copy_wait<C::AHEAD>();
                phases ^= 1u << b;
                __syncwarp();
            }
            if (!ok) break;
            tc_fence_after();
            if (mine) {
                const uint32_t from = tmem + acc * C::TN + half * (C::TN / 2) + ((uint32_t)(quarter * 32) << 16);
#pragma unroll
                for (int c = 0; c < C::TN / 2; c += 32) {
                    uint32_t d[32];
                    tmem_ld_32x32b_x32(from + c, d);
                    uint8_t *row = box(b, c / C::PER) + lane * 128;
                    const int first = c % C::PER * C::ELEM / 16;
                    auto at = [&](int j) { return reinterpret_cast<uint4 *>(row + (((first + j) ^ (lane & 7)) << 4)); };
                    uint4 old[2 * C::ELEM];
#pragma unroll
                    for (int j = 0; j < 2 * C::ELEM; ++j) old[j] = base ? *at(j) : make_uint4(0, 0, 0, 0);
                    tmem_ld_wait(d);
#pragma unroll
                    for (int j = 0; j < 2 * C::ELEM; ++j) {
                        const uint4 o = old[j];
                        if constexpr (C::ELEM == 2) {
                            auto add = [&](uint32_t two, int k) {
                                const __nv_bfloat162 v = __floats2bfloat162_rn(lo_f32(two) + __uint_as_float(d[k]), hi_f32(two) + __uint_as_float(d[k + 1]));
                                return *reinterpret_cast<const uint32_t *>(&v);
                            };
                            *at(j) = make_uint4(add(o.x, 8 * j), add(o.y, 8 * j + 2), add(o.z, 8 * j + 4), add(o.w, 8 * j + 6));
                        } else {
                            auto add = [&](uint32_t one, int k) { return __float_as_uint(__uint_as_float(one) + __uint_as_float(d[k])); };
                            *at(j) = make_uint4(add(o.x, 4 * j), add(o.y, 4 * j + 1), add(o.z, 4 * j + 2), add(o.w, 4 * j + 3));
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&t_empty[acc]);
            if (mine && packed && left >= 32) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    for (int x = 0; x < C::OWN; ++x)
                        if (column(nt, x) < p.C) tma_store_2d(&om, smem_u32(box(b, x)), column(nt, x), token);
                    bulk_commit_group();
                }
            } else if (mine) {
                for (int x = 0; x < C::OWN; ++x) {
                    const int col = column(nt, x), n = chunks(col);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int r = k * 4 + (lane >> 3), t = __shfl_sync(0xffffffffu, token, r);
                        if (t >= 0 && (lane & 7) < n)
                            *place(out, t, col, lane & 7) = *reinterpret_cast<const uint4 *>(box(b, x) + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
                    }
                }
                if (packed) fence_proxy_async_smem();        // (the next base comes by TMA)
                __syncwarp();
            }
            b = b + 1 == C::NB ? 0 : b + 1;
        }
        if (!ok && mine && base && packed && lane == 0)      // (a launch that gave up: no copy is left on its way)
            for (int k = i; k <= i + C::AHEAD; ++k)
                if (g + k * G < n_tiles) mbar_wait(&b_full[warp * C::NB + k % C::NB], (k / C::NB) & 1, nullptr, p.err);
        copy_wait<0>();
        if (lane == 0) bulk_wait_group_all();
        __syncwarp();
    } else if (any && warp == E_WARPS) {
        // v's pieces, K-major, the three one after another
        const uint32_t idesc = idesc_bf16_f32(128, C::TN, false, C::MN), sv = smem_u32(smem), sw = sv + C::OFF_W;
        const int steps = r16 / 16;
        if (lane == 0) {
            const int boxes = pieces_pitch(p.r) / 64;
            mbar_arrive_expect_tx(v_full, boxes * 16384);
            for (int x = 0; x < boxes; ++x) tma_load_2d(smem + x * 16384, &vm, v_full, x * 64, wk.row0);
        }
        __syncwarp();
        int i = 0;
        bool ok = bar_wait_warp(v_full, 0, abort_flag, p.err);
        for (int nt = g; ok && nt < n_tiles; nt += G, ++i) {
            const int b = i & 1;
            ok = bar_wait_warp(&w_full[b], (i >> 1) & 1, abort_flag, p.err) &&
                 (i < 2 || bar_wait_warp(&t_empty[b], ((i >> 1) & 1) ^ 1, abort_flag, p.err));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                for (int k = 0; k < steps; ++k) {
                    const uint32_t wb = sw + b * C::W_BYTES;
                    const uint64_t wd = C::MN ? smem_desc_mn_sw128(wb, r16 * 128) + k * k_step(true)
                                              : smem_desc_k_sw128(wb + (k >> 2) * C::TN * 128) + (k & 3) * k_step(false);
#pragma unroll
                    for (int q = 0; q < 3; ++q) {
                        const int a = q * steps + k;
                        tc_mma_bf16(tmem + b * C::TN, smem_desc_k_sw128(sv + (a >> 2) * 16384) + (a & 3) * k_step(false), wd, idesc, (k | q) != 0);
                    }
                }
                tc_commit(&w_empty[b]);
                tc_commit(&t_full[b]);
            }
            __syncwarp();
            if (nt + 2 * G < n_tiles) {                      // (once W's tile has been read)
                ok = bar_wait_warp(&w_empty[b], (i >> 1) & 1, abort_flag, p.err);
                if (!ok) break;
                if (lane == 0) load_w(nt + 2 * G, b);
                __syncwarp();
            }
        }
        if (!ok) {
            // (a launch that gave up: no copy and nothing issued is left on its way; waits for
            // what was not begun end at their bound)
            mbar_wait(v_full, 0, nullptr, p.err);
            for (int k = 0; k < 2; ++k) {
                mbar_wait(&w_full[k], ((i + (k != (i & 1))) >> 1) & 1, nullptr, p.err);
                if (i > 1) mbar_wait(&w_empty[k], ((i - 1 - (k != ((i - 1) & 1))) >> 1) & 1, nullptr, p.err);
            }
        }
        __syncwarp();
    } else if (warp > E_WARPS && out != base) {
        // tokens of no adapter keep base
        // (a warp looks at 32 at once: one after another, 32768 tokens of 8 adapters, which is to
        // say none to copy, took 149 us instead of 83)
        const int64_t per = (p.T + gridDim.x * 3 - 1) / (gridDim.x * 3);
        const int first = (int)min((int64_t)p.T, (blockIdx.x * 3 + warp - E_WARPS - 1) * per), end = (int)min((int64_t)p.T, first + per);
        for (int q0 = first; q0 < end; q0 += 32) {
            const int q = q0 + lane;
            unsigned none = __ballot_sync(0xffffffffu, q < end && (unsigned)__ldcg(p.slot_row + min(q, p.T - 1)) >= (unsigned)p.T);
            for (; none; none &= none - 1) {
                const int64_t at = (q0 + __ffs(none) - 1) * pitch;
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(base) + at);
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(out) + at);
                for (int c = lane; c < (int)(pitch / 16); c += 32 * 4) {
                    uint4 f[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) f[j] = base && c + 32 * j < (int)(pitch / 16) ? __ldcg(src + c + 32 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (c + 32 * j < (int)(pitch / 16)) dst[c + 32 * j] = f[j];
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == E_WARPS) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// Outer products on the tensor cores: a tile is 128 columns of x (on the MMA's M side, as
// they lie in memory) times v's three pieces side by side (one MMA reads x once for all
// three: with one for each piece their reads of x were the bound), summed over an adapter's
// rows, 64 a stage.  Persistent; where tensor memory has room for two accumulators (r up to
// 80) one is taken out while the next tile's MMAs run.  Rows as in shrink: by TMA where
// their tokens follow one another, but for an adapter's last ones.  4096 rows of 4096 and of 11008
// columns, 4 adapters, r = 32: 38 us for both, 3.2 TB/s; 3.1 rounds of tiles take four.
//
// Roles: warp 0 loads by TMA, warp 2 issues the MMAs, warps 4 .. 11 gather what TMA does not,
// warps 12 .. 15 take a tile out (32 columns of x each).
// ---------------------------------------------------------------------------
constexpr int O_THREADS = 512;
// Stages of a part, as a logarithm: the tensor core's adds drop what is below the accumulator's last
// bit (positive values: of 512 2.3e-7 short, of 4096 7.9e-6), so that 512 tokens at most are summed
// there.  The sum of the parts before is in tensor memory behind the first accumulator's columns.
// Of bf16 results, whose rounding is 4e-3, 4096 where only one accumulator has room beside that
// sum (16384 tokens, r = 128: 359 us a gradient, in parts of 512 395; r = 64 250 / 251).
constexpr int PART_LOG = 3, LONG_PART_LOG = 6;

template <int BOXES_>
struct OuterCfg {
    static constexpr int BOXES = BOXES_;                     // 64-wide boxes of the pieces, at most: 2 (r up to 32), 4 (80), 6
    static constexpr bool WIDE = BOXES > 4;
    static constexpr int STAGE = 16384 + BOXES * 8192;
    static constexpr int NS = BOXES == 2 ? 6 : BOXES == 4 ? 4 : 3, LAG = NS - 1;
    static constexpr int ACC = WIDE ? 1 : 2, ACC_COLS = 512 / ACC;
    static constexpr int OFF_BAR = NS * STAGE;
    static constexpr int SMEM = 1024 + OFF_BAR + (2 * NS + 4) * 8 + 8;
};

// d [L][r][C], or (transposed) [L][C][r].  A launch has two: an adapter's tiles are the first
// one's and then the second one's.
struct OuterJob {
    CUtensorMap xm, vm;
    const __nv_bfloat16 *x, *v16;
    void *d;
    int C, n_tiles, wide_x, transposed;
};

template <class C>
__global__ void __launch_bounds__(O_THREADS, 1) outer_kernel(const __grid_constant__ OuterJob ja, const __grid_constant__ OuterJob jb, const Params p,
                                                             int d_bf16, int part_log) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *s_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *s_empty = s_full + C::NS, *t_full = s_empty + C::NS, *t_empty = t_full + 2;
    int *info = reinterpret_cast<int *>(t_empty + 2);        // abort, TMEM base
    volatile int *abort_flag = info;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    const int r16 = up16(p.r), part_mask = (1 << part_log) - 1;
    if (tid == 0) {
        info[0] = 0;
        for (int i = 0; i < C::NS; ++i) { mbar_init(&s_full[i], 9); mbar_init(&s_empty[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&t_full[i], 1); mbar_init(&t_empty[i], 4); }
        fence_mbarrier_init();
        prefetch_tensormap(&ja.xm);
        prefetch_tensormap(&ja.vm);
        prefetch_tensormap(&jb.xm);
        prefetch_tensormap(&jb.vm);
    }
    if (warp == 2) {
        tmem_alloc(reinterpret_cast<uint32_t *>(info + 1), 512);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    grid_wait();
    grid_launch_dependents();          // (this block has its tensor memory)
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(info + 1);
    GroupWalk<128, 1, true> wk;
    if (warp != 1 && warp != 3) wk.start(p.offsets, p.T, p.L, ja.n_tiles + jb.n_tiles, p.each, false, blockIdx.x);
    auto stages = [&] { return (wk.rows + KB - 1) / KB; };
    // The tile's stages that TMA loads, the first ones: all whole ones where the group's tokens
    // follow one another, else none (looked at again only where the group has changed).
    int whole_of = -1, whole = 0;
    auto whole_stages = [&] {
        if (wk.e == whole_of) return whole;
        bool packed = wk.rows >= KB;
        const int32_t *slot = p.row_slot + wk.row0;
        const int t0 = packed ? __ldcg(slot) : -1;
        packed = packed && t0 >= 0 && t0 <= p.T - wk.rows;
        // (all loads of 1024 rows on their way: one after another, ending at the first stranger,
        // they took three quarters of the kernel's time, in eights a sixth)
        for (int i = lane; packed && i < wk.rows; i += 32 * 32) {
            int t[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) t[j] = i + 32 * j < wk.rows ? __ldcg(slot + i + 32 * j) : t0 + i + 32 * j;
#pragma unroll
            for (int j = 0; j < 32; ++j) packed = packed && t[j] == t0 + i + 32 * j;
        }
        whole_of = wk.e;
        whole = __all_sync(0xffffffffu, packed) ? wk.rows / KB : 0;
        return whole;
    };

    if (warp == 0) {
        // ---- by TMA
        const int boxes = pieces_pitch(p.r) / 64;
        uint32_t it = 0, asked = 0;                          // asked: the stages whose last fill was this warp's
        bool ok = true;
        for (; ok && wk.get(); wk.t += gridDim.x) {
            const int ns = stages(), n = whole_stages(), t0 = n ? __ldcg(p.row_slot + wk.row0) : 0;
            const OuterJob &job = wk.nt < ja.n_tiles ? ja : jb;
            const int nt = wk.nt < ja.n_tiles ? wk.nt : wk.nt - ja.n_tiles;
            // (This warp and the gathering ones each arrive for every stage, whoever fills it: who
            // only waited for s_empty could be left more than a phase behind, and a barrier
            // tells a phase from the next one alone.)
            for (int i = 0; i < ns; ++i, ++it) {
                const uint32_t s = it % C::NS;
                if (it >= (uint32_t)C::NS) ok = bar_wait_warp(&s_empty[s], ((it / C::NS) & 1) ^ 1, abort_flag, p.err);
                if (!ok) break;
                if (i >= n) {
                    asked &= ~(1u << s);
                    if (lane == 0) mbar_arrive(&s_full[s]);
                    __syncwarp();
                    continue;
                }
                asked |= 1u << s;
                uint8_t *to = smem + s * C::STAGE;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&s_full[s], 16384 + boxes * 8192);
                    if (job.wide_x) {
                        tma_load_3d(to, &job.xm, &s_full[s], 0, t0 + i * KB, nt * 2);
                    } else {
                        tma_load_2d(to, &job.xm, &s_full[s], nt * 128, t0 + i * KB);
                        tma_load_2d(to + 8192, &job.xm, &s_full[s], nt * 128 + 64, t0 + i * KB);
                    }
                    tma_load_3d(to + 16384, &job.vm, &s_full[s], 0, wk.row0 + i * KB, 0);
                }
                __syncwarp();
            }
        }
        if (lane == 0 && *abort_flag)                        // no copy is left on its way
            for (uint32_t j = it > (uint32_t)C::NS ? it - C::NS : 0; j < it; ++j)
                if ((asked >> (j % C::NS)) & 1) mbar_wait(&s_full[j % C::NS], (j / C::NS) & 1, nullptr, p.err);
        __syncwarp();
    } else if (warp >= 4 && warp < 12) {
        // ---- gather: x's rows (thread = one 16-byte column of rows me / 16 + 16 j) and the
        // pieces' (16-byte columns in turn); zeros past the group's rows and for rows of no token
        const int me = tid - 128, chunk = me & 15, first = me >> 4, wide = 3 * r16 / 8;
        const uint32_t dst = smem_u32(smem) + (chunk >> 3) * 8192 + first * 128 + (((chunk & 7) ^ (first & 7)) << 4);
        const FastDiv by_wide = p.by_wide;
        uint32_t it = 0, sent = 0, mine = 0;                 // mine: a bit for each stage
        bool ok = true;
        auto filled = [&] {            // this thread's copies of the oldest stage have arrived
            const uint32_t s = sent % C::NS;
            if ((mine >> s) & 1) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_full[s]);
            }
            ++sent;
        };
        for (; ok && wk.get(); wk.t += gridDim.x) {
            const int ns = stages(), n = whole_stages();
            const OuterJob &job = wk.nt < ja.n_tiles ? ja : jb;
            const int col = (wk.nt < ja.n_tiles ? wk.nt : wk.nt - ja.n_tiles) * 128 + chunk * 8;
            // tokens of rows lane and 32 + lane of a stage, asked for a stage ahead
            int t[2];
            auto tokens = [&](int i) {
#pragma unroll
                for (int j = 0; j < 2; ++j) t[j] = i * KB + j * 32 + lane < wk.rows ? __ldcg(p.row_slot + wk.row0 + i * KB + j * 32 + lane) : -1;
            };
            if (n < ns) tokens(n);
            for (int i = 0; i < ns; ++i, ++it) {
                const uint32_t s = it % C::NS;
                mine &= ~(1u << s);
                if (i < n) {
                    if (it >= (uint32_t)C::NS) ok = bar_wait_warp(&s_empty[s], ((it / C::NS) & 1) ^ 1, abort_flag, p.err);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive(&s_full[s]);
                } else {
                    mine |= 1u << s;
                    if (it >= (uint32_t)C::NS) ok = bar_wait_warp(&s_empty[s], ((it / C::NS) & 1) ^ 1, abort_flag, p.err);
                    if (!ok) break;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int tok = __shfl_sync(0xffffffffu, t[j >> 1], (first + 16 * j) & 31);
                        const bool there = (unsigned)tok < (unsigned)p.T && col < job.C;
                        copy16(dst + s * C::STAGE + j * 2048, there ? job.x + (int64_t)tok * job.C + col : job.x, there);
                    }
                    const uint32_t to = smem_u32(smem) + s * C::STAGE + 16384;
                    const int pieces = min(KB, (wk.rows - i * KB + 15) / 16 * 16) * wide;   // (rows past those: no MMA takes)
                    for (int q0 = 0; q0 < pieces; q0 += 256) {
                        const int q = q0 + me, row = min(by_wide.div(q), KB - 1), c = q - row * wide;
                        const int t0 = __shfl_sync(0xffffffffu, t[0], row & 31), t1 = __shfl_sync(0xffffffffu, t[1], row & 31);
                        const bool there = (unsigned)(row < 32 ? t0 : t1) < (unsigned)p.T;
                        if (q < pieces)
                            copy16(to + (c >> 3) * 8192 + row * 128 + (((c & 7) ^ (row & 7)) << 4),
                                   there ? job.v16 + (int64_t)(wk.row0 + i * KB + row) * pieces_pitch(p.r) + c * 8 : job.v16, there);
                    }
                    if (i + 1 < ns) tokens(i + 1);
                }
                copy_commit();
                if (it - sent >= (uint32_t)C::LAG) {
                    copy_wait<C::LAG>();
                    filled();
                }
            }
        }
        copy_wait<0>();
        if (ok)
            while (sent != it) filled();
    } else if (warp == 2) {
        // ---- MMA issuer: columns 0 .. 255 of the pieces, and those past them
        const int cols = 3 * r16, low = cols < 256 ? cols : 256;
        const uint32_t idesc = idesc_bf16_f32(128, low, true, true), idesc_high = idesc_bf16_f32(128, cols > 256 ? cols - 256 : 16, true, true);
        const bool high = C::WIDE && cols > 256;
        uint32_t it = 0, acc = 0;
        bool ok = true;
        for (; ok && wk.get(); wk.t += gridDim.x) {
            const int ns = stages();
            if (ns == 0) continue;
            for (int i = 0; i < ns; ++i, ++it) {
                const uint32_t s = it % C::NS, b = acc % C::ACC, dst = tmem + b * C::ACC_COLS;
                const int at = i & part_mask;                // a part's first stage: 0
                const bool last = at == part_mask || i == ns - 1;
                if (at == 0) ok = acc < (uint32_t)C::ACC || bar_wait_warp(&t_empty[b], ((acc / C::ACC) & 1) ^ 1, abort_flag, p.err);
                ok = ok && bar_wait_warp(&s_full[s], (it / C::NS) & 1, abort_flag, p.err);
                if (!ok) break;
                tc_fence_after();
                const uint32_t sx = smem_u32(smem) + s * C::STAGE, sv = sx + 16384;
                const int n = (min(KB, wk.rows - i * KB) + 15) / 16;
                const uint64_t xd = smem_desc_mn_sw128(sx, 8192), vd = smem_desc_mn_sw128(sv, 8192), vh = smem_desc_mn_sw128(sv + 4 * 8192, 8192);
                if (elect_one()) {
                    for (int k = 0; k < n; ++k) {
                        tc_mma_bf16(dst, xd + k * k_step(true), vd + k * k_step(true), idesc, (at | k) != 0);
                        if (high) tc_mma_bf16(dst + 256, xd + k * k_step(true), vh + k * k_step(true), idesc_high, (at | k) != 0);
                    }
                    tc_commit(&s_empty[s]);
                    if (last) tc_commit(&t_full[b]);
                }
                __syncwarp();
                acc += last;
            }
            ok = __all_sync(0xffffffffu, ok && !*abort_flag);
        }
        // (what was issued is waited for by the warps that take it out; a launch that gave up
        // waits here, on a barrier that nothing else arrives on any more)
        if (!ok && it > 0) {
            if (lane == 0) mbar_wait(&s_empty[(it - 1) % C::NS], ((it - 1) / C::NS) & 1, nullptr, p.err);
            __syncwarp();
        }
    } else if (warp >= 12) {
        // ---- take out, add the three pieces' sums, write: thread = one column of x
        const uint32_t from = tmem + ((uint32_t)((warp & 3) * 32) << 16), sums = from + 3 * r16;   // of the parts before
        uint32_t acc = 0;
        for (bool ok = true; ok && wk.get(); wk.t += gridDim.x) {
            const int parts = (stages() + part_mask) >> part_log;
            const bool some = parts > 0;
            const OuterJob &job = wk.nt < ja.n_tiles ? ja : jb;
            const int c = (wk.nt < ja.n_tiles ? wk.nt : wk.nt - ja.n_tiles) * 128 + (warp & 3) * 32 + lane;
            void *d = job.d;
            for (int i = 0; i == 0 || i < parts; ++i) {
                const uint32_t b = acc % C::ACC;
                if (some) {
                    ok = bar_wait_warp(&t_full[b], (acc / C::ACC) & 1, abort_flag, p.err);
                    if (!ok) break;
                    tc_fence_after();
                    ++acc;
                }
                for (int j0 = 0; j0 < p.r; j0 += 16) {
                    uint32_t w[16];
                    if (some) {
                        uint32_t w1[16], w2[16];
                        tmem_ld_32x32b_x16(from + b * C::ACC_COLS + j0, w);
                        tmem_ld_32x32b_x16(from + b * C::ACC_COLS + r16 + j0, w1);
                        tmem_ld_32x32b_x16(from + b * C::ACC_COLS + 2 * r16 + j0, w2);
                        tmem_ld_wait(w);
                        tmem_ld_wait(w1);
                        tmem_ld_wait(w2);
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(__uint_as_float(w[j]) + (__uint_as_float(w1[j]) + __uint_as_float(w2[j])));
                        if (i > 0) {
                            tmem_ld_32x32b_x16(sums + j0, w1);
                            tmem_ld_wait(w1);
#pragma unroll
                            for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(__uint_as_float(w1[j]) + __uint_as_float(w[j]));
                        }
                        if (i < parts - 1) {
                            tmem_st_32x32b_x16(sums + j0, w);
                            continue;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[j] = 0;
                    }
                    if (c >= job.C) continue;
                    if (job.transposed) {  // d [L][C][r]
                        const int64_t at = ((int64_t)wk.e * job.C + c) * p.r + j0;
#pragma unroll
                        for (int j = 0; j < 16; j += 8) {
                            if (j0 + j >= p.r) break;
                            if (d_bf16) {
                                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(d) + at + j) =
                                    make_uint4(bf16x2(w[j], w[j + 1]), bf16x2(w[j + 2], w[j + 3]), bf16x2(w[j + 4], w[j + 5]), bf16x2(w[j + 6], w[j + 7]));
                            } else {
                                *reinterpret_cast<uint4 *>(static_cast<float *>(d) + at + j) = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
                                *reinterpret_cast<uint4 *>(static_cast<float *>(d) + at + j + 4) = make_uint4(w[j + 4], w[j + 5], w[j + 6], w[j + 7]);
                            }
                        }
                    } else {               // d [L][r][C]
                        const int64_t at = ((int64_t)wk.e * p.r + j0) * job.C + c;
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            if (j0 + j >= p.r) break;
                            if (d_bf16) static_cast<__nv_bfloat16 *>(d)[at + (int64_t)j * job.C] = __float2bfloat16_rn(__uint_as_float(w[j]));
                            else static_cast<float *>(d)[at + (int64_t)j * job.C] = __uint_as_float(w[j]);
                        }
                    }
                }
                if (some) {
                    if (i < parts - 1) tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&t_empty[b]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// Few tokens (decoding requests): one block for a token's row and some rows of W, sums in
// fp32 by the ordinary units.
// ---------------------------------------------------------------------------

// The group of `row`: the last offset up to the first one above it; L: none, -1: before
// the first.  The whole block; `sh`: a word of shared memory.
__device__ __forceinline__ int group_of(const int32_t *offsets, int L, int T, int row, int *sh) {
    if (threadIdx.x == 0) *sh = L + 1;
    __syncthreads();
    int first = L + 1;
    for (int g = threadIdx.x; g <= L && first > L; g += 4 * blockDim.x) {
        int o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __ldcg(offsets + min(L, g + i * (int)blockDim.x));
#pragma unroll
        for (int i = 3; i >= 0; --i)
            if (o[i] > row) first = min(L, g + i * (int)blockDim.x);
    }
    first = __reduce_min_sync(0xffffffffu, first);
    if ((threadIdx.x & 31) == 0 && first <= L) atomicMin(sh, first);
    __syncthreads();
    return *sh - 1;
}

__device__ __forceinline__ float dot8(uint4 a, uint4 b, float s) {
    s = fmaf(lo_f32(a.x), lo_f32(b.x), s); s = fmaf(hi_f32(a.x), hi_f32(b.x), s);
    s = fmaf(lo_f32(a.y), lo_f32(b.y), s); s = fmaf(hi_f32(a.y), hi_f32(b.y), s);
    s = fmaf(lo_f32(a.z), lo_f32(b.z), s); s = fmaf(hi_f32(a.z), hi_f32(b.z), s);
    s = fmaf(lo_f32(a.w), lo_f32(b.w), s); s = fmaf(hi_f32(a.w), hi_f32(b.w), s);
    return s;
}

// PARTS warps for one value of v: blocks (row, 8 of r).  Two where the blocks are few (61 tokens
// of 48 adapters, K = 4096, r = 16, with expand, calls chained in a graph: 8.9 us, one warp 10.3); of
// many blocks they cost more than they gain (128 of 64, r = 64: one warp 50.5 us, two some 3 more).
template <int PARTS>
__global__ void __launch_bounds__(256 * PARTS) shrink_row_kernel(const Params p, const __nv_bfloat16 *x, const __nv_bfloat16 *w, float *v) {
    __shared__ int sh;
    __shared__ float sums[8 * PARTS];
    grid_wait();
    grid_launch_dependents();
    const int row = blockIdx.x, warp = threadIdx.x >> 5, part = warp >> 3, j = blockIdx.y * 8 + (warp & 7), lane = threadIdx.x & 31;
    const int t = __ldcg(p.row_slot + row);
    const int e = group_of(p.offsets, p.L, p.T, row, &sh);
    if (e < 0) return;
    float sum = 0.0f;
    if (e < p.L && (unsigned)t < (unsigned)p.T) {
        const uint4 *a = reinterpret_cast<const uint4 *>(x + (int64_t)t * p.C);
        const uint4 *b = reinterpret_cast<const uint4 *>(w + ((int64_t)e * p.r + j) * p.C);
        const int each = (p.C / 8 + PARTS - 1) / PARTS, n = min(p.C / 8, each * (part + 1));
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        int c = each * part + lane;
        for (; c + 7 * 32 < n; c += 8 * 32) {
            uint4 fa[8], fb[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) { fb[i] = __ldcg(b + c + i * 32); fa[i] = __ldcg(a + c + i * 32); }
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i & 3] = dot8(fa[i], fb[i], s[i & 3]);
        }
        for (; c < n; c += 32) s[0] = dot8(__ldcg(a + c), __ldcg(b + c), s[0]);
        sum = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if constexpr (PARTS > 1) {
        if (lane == 0) sums[warp] = sum;
        __syncthreads();
        if (part) return;
        for (int k = 1; k < PARTS; ++k) sum += sums[warp + 8 * k];
    }
    if (lane == 0) v[(int64_t)row * p.r + j] = p.scale && e < p.L ? sum * __ldcg(p.scale + e) : sum;
}

constexpr int R_THREADS = 128;

// Two columns of out a thread: blocks (token, 256 columns).  W's rows and base are asked for
// before the grid that writes v has ended, and from L2: this SM's L1 may hold what was there
// before the grids before that one (through L1, which gives the other half of a row's 32 bytes,
// 61 tokens of 48 adapters with r = 16 took 0.6 us less).
template <typename O>
__global__ void __launch_bounds__(R_THREADS) expand_row_kernel(const Params p, const float *v, const __nv_bfloat16 *w, const O *base, O *out) {
    __shared__ int sh;
    __shared__ __align__(16) float vs[128];   // (read 16 bytes at a time)
    const int t = blockIdx.x, n = blockIdx.y * (2 * R_THREADS) + threadIdx.x * 2, row = __ldcg(p.slot_row + t);
    const bool some = (unsigned)row < (unsigned)p.T;
    const int e = some ? group_of(p.offsets, p.L, p.T, row, &sh) : p.L;
    const bool there = n < p.C;        // (C is a multiple of 8)
    const int64_t at = (int64_t)t * p.C + n;
    float a = 0.0f, b = 0.0f;
    if (there && base) {
        if constexpr (sizeof(O) == 2) {
            const uint32_t two = __ldcg(reinterpret_cast<const uint32_t *>(base + at));
            a = lo_f32(two), b = hi_f32(two);
        } else {
            const float2 two = __ldcg(reinterpret_cast<const float2 *>(base + at));
            a = two.x, b = two.y;
        }
    }
    constexpr int AHEAD = 4;
    const uint4 *w0 = reinterpret_cast<const uint4 *>(w + ((int64_t)e * p.C + n) * p.r), *w1 = w0 + p.r / 8;
    const bool mine = there && e >= 0 && e < p.L;
    uint4 f[2][AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (mine && i * 8 < p.r) { f[0][i] = __ldcg(w0 + i); f[1][i] = __ldcg(w1 + i); }
    grid_wait();
    grid_launch_dependents();
    if (e >= 0 && e < p.L) {
        for (int i = threadIdx.x; i < p.r; i += R_THREADS) vs[i] = __ldcg(v + (int64_t)row * p.r + i);
        __syncthreads();
    }
    if (mine) {
        auto dot = [&](uint4 q, int c, float s) {
            const float4 lo = *reinterpret_cast<const float4 *>(vs + c), hi = *reinterpret_cast<const float4 *>(vs + c + 4);
            s = fmaf(lo_f32(q.x), lo.x, s); s = fmaf(hi_f32(q.x), lo.y, s); s = fmaf(lo_f32(q.y), lo.z, s); s = fmaf(hi_f32(q.y), lo.w, s);
            s = fmaf(lo_f32(q.z), hi.x, s); s = fmaf(hi_f32(q.z), hi.y, s); s = fmaf(lo_f32(q.w), hi.z, s); s = fmaf(hi_f32(q.w), hi.w, s);
            return s;
        };
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (i * 8 < p.r) { s0 = dot(f[0][i], i * 8, s0); s1 = dot(f[1][i], i * 8, s1); }
        for (int i = AHEAD; i * 8 < p.r; ++i) { s0 = dot(__ldcg(w0 + i), i * 8, s0); s1 = dot(__ldcg(w1 + i), i * 8, s1); }
        a += s0;
        b += s1;
    }
    if (there && (mine || out != base)) {
        if constexpr (sizeof(O) == 2) *reinterpret_cast<__nv_bfloat162 *>(out + at) = __floats2bfloat162_rn(a, b);
        else *reinterpret_cast<float2 *>(out + at) = make_float2(a, b);
    }
}

// The same where r / 8 is a power of two, q: lane l of a load of 512 bytes of W's rows takes 16
// of them, ranks 8 (l % q) and on of column l / q, whose sums the q lanes join.  A block takes
// several runs of columns where the blocks are many more than run at once (4096 -> 11008, calls
// chained in a graph, with shrink: 61 tokens of 48 adapters, r = 16, 8.9 us, by two columns a thread
// 10.1; 512 of 64 43.9 / 67.5; 128 of 64, r = 64, 50.5 / 58.4).
template <typename O>
__global__ void __launch_bounds__(R_THREADS) expand_lane_kernel(const Params p, const float *v, const __nv_bfloat16 *w, const O *base, O *out, int q_log) {
    __shared__ int sh;
    constexpr int LOADS = 8;
    const int t = blockIdx.x, lane = threadIdx.x & 31, q = 1 << q_log, k = lane & (q - 1), row = __ldcg(p.slot_row + t);
    const int e = (unsigned)row < (unsigned)p.T ? group_of(p.offsets, p.L, p.T, row, &sh) : p.L;
    const bool mine = e >= 0 && e < p.L;
    const int all = p.C << q_log, step = gridDim.y * (R_THREADS * LOADS);     // 16-byte pieces of W[e]
    const uint4 *from = reinterpret_cast<const uint4 *>(w) + (int64_t)e * all;
    const O *old = base + (int64_t)t * p.C;
    O *to = out + (int64_t)t * p.C;
    float vs[8];
    bool waited = false;
    for (int c0 = (blockIdx.y * (R_THREADS / 32) + (threadIdx.x >> 5)) * (32 * LOADS); !waited || c0 < all; c0 += step) {
        uint4 f[LOADS];
        float b[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int c = c0 + i * 32 + lane;
            f[i] = mine && c < all ? __ldcg(from + c) : make_uint4(0, 0, 0, 0);
            b[i] = 0.0f;
            if (base && (i & (q - 1)) == k && c < all) {
                if constexpr (sizeof(O) == 2) b[i] = __uint_as_float((uint32_t)__ldcg(reinterpret_cast<const uint16_t *>(old) + (c >> q_log)) << 16);
                else b[i] = __ldcg(old + (c >> q_log));
            }
        }
        if (!waited) {
            grid_wait();
            grid_launch_dependents();
            if (mine) {
                const float4 lo = __ldcg(reinterpret_cast<const float4 *>(v + (int64_t)row * p.r + k * 8)), hi = __ldcg(reinterpret_cast<const float4 *>(v + (int64_t)row * p.r + k * 8 + 4));
                vs[0] = lo.x; vs[1] = lo.y; vs[2] = lo.z; vs[3] = lo.w;
                vs[4] = hi.x; vs[5] = hi.y; vs[6] = hi.z; vs[7] = hi.w;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) vs[i] = 0.0f;
            }
            waited = true;
        }
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            float s = lo_f32(f[i].x) * vs[0];
            s = fmaf(hi_f32(f[i].x), vs[1], s); s = fmaf(lo_f32(f[i].y), vs[2], s); s = fmaf(hi_f32(f[i].y), vs[3], s);
            s = fmaf(lo_f32(f[i].z), vs[4], s); s = fmaf(hi_f32(f[i].z), vs[5], s); s = fmaf(lo_f32(f[i].w), vs[6], s); s = fmaf(hi_f32(f[i].w), vs[7], s);
#pragma unroll
            for (int o = 1; o < 16; o <<= 1)
                if (o < q) s += __shfl_xor_sync(0xffffffffu, s, o);
            const int c = c0 + i * 32 + lane;
            if ((i & (q - 1)) == k && c < all && (mine || out != base)) {   // (of the q lanes that have the sum one)
                const float y = mine ? b[i] + s : b[i];
                if constexpr (sizeof(O) == 2) to[c >> q_log] = __float2bfloat16_rn(y);
                else to[c >> q_log] = y;
            }
        }
    }
}

// ---- host -------------------------------------------------------------------

static Params params(const LoraPlan &q, int C) { return Params{q.row_slot, q.slot_row, q.offsets, q.scale, q.err, q.T, q.r, q.L, C, FastDiv(1), FastDiv(up16(q.r) / 4), FastDiv(3 * up16(q.r) / 8)}; }
// Row tiles of 128 rows, at most, with those of the rows of none.
static int64_t row_tiles(const LoraPlan &q) { return q.T / 128 + (q.L + 1 < q.T ? q.L + 1 : q.T); }
// Whether a forward pass goes row by row: each row reads its adapter through L2 again, where
// the tensor cores' kernels take a tile for each adapter, however few its rows.  L is the table's
// size; how many adapters have tokens the host does not know, and by tiles that decides: the bound
// lies where neither form is much more than twice the other, whether one adapter has all tokens or
// each has some (4096 -> 11008, us by rows and by tiles with one in use / all: 128 tokens of 8 adapters, r =
// 16: 13 and 10 / 20; 24 of 8, r = 128: 21 and 16 / 26; 256 of 16, r = 16: 21 and 12 / 27; 40 of 32, r = 128: 28 to
// 30 and 19 / 43; 512 of 32, r = 16: 39 and 15 / 45; 512 of 64, r = 16: 41 and 18 / 79; 1024 of 128, r = 16: 75 to
// 85 and 27 / 150; 512 of 128, r = 32: 78 to 95 and 25 / 144; 1024 of 256, r = 32: 157 to 171 and 108 / 276; 2048
// of 256, r = 32: 282 to 303 and 111 / 285; 2048 of 1024, r = 64: 550 to 647 and 243 / 893; 16384 of 4096, r =
// 16: 1050 to 1310 and 2916 / 4826, whose walk over the table each block takes).  r = 24 and the like, two
// columns a thread, take a third longer and more by rows (100 of 32, r = 40: 29 to 32 and 12 / 44; 512 of
// 128, r = 24: 91 to 121 and 25 / 144).
static bool lane_wide(int r) { return (r & (r - 1)) == 0; }   // r is a multiple of 8
static bool few(int T, int r, int L) {
    const int64_t in_use = L < T ? L : T;                     // adapters, at most
    return (int64_t)T * r <= (lane_wide(r) ? 1700 + 104 * in_use : 1400 + 62 * in_use);
}

template <bool MN>
static cudaError_t shrink(const LoraPlan &q, const void *x, const void *w, float *v, void *v16, const float *other, void *other16, int C, cudaStream_t s) {
    CUtensorMap rows, map;
    if (!encode(&rows, x, 2, C, q.T, 1, 128, false)) return cudaErrorInvalidValue;
    if (!(MN ? encode(&map, w, 2, q.r, C, q.L, KB, true) : encode(&map, w, 2, C, q.r, q.L, q.r, true))) return cudaErrorInvalidValue;
    const DeviceInfo &di = device_info();
    // few tiles: the contraction over as many blocks as run at once, two stages each at least
    const int64_t tiles = row_tiles(q);
    const int blocks = (C + KB - 1) / KB;
    int split = S_MAX_SPLIT;
    while (split > 1 && (tiles * split > di.num_sms * (s_smem(q.r, MN) <= 113 * 1024 ? 2 : 1) || blocks < 2 * split)) split /= 2;
    const size_t smem = s_smem(q.r, MN);
    const cudaError_t e = ensure_dynamic_smem((const void *)shrink_kernel<MN>, smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(shrink_kernel<MN>, dim3((unsigned)(tiles * split)), S_THREADS, smem, (unsigned)split, s, rows, map, params(q, C),
                            static_cast<const __nv_bfloat16 *>(x), v, static_cast<__nv_bfloat16 *>(v16), other, static_cast<__nv_bfloat16 *>(other16));
}

template <int ELEM, int TN, int BOXES, bool MN>
static cudaError_t expand(const LoraPlan &q, const void *v16, const void *w, const void *base, void *out, int C, cudaStream_t s) {
    using Cfg = ExpandCfg<ELEM, TN, BOXES, MN>;
    CUtensorMap rows, map, from{}, to;
    if (!encode(&rows, v16, 2, pieces_pitch(q.r), q.T, 1, 128, false) || !encode(&to, out, ELEM, C, q.T, 1, 32, false)) return cudaErrorInvalidValue;
    if (base && !encode(&from, base, ELEM, C, q.T, 1, 32, false)) return cudaErrorInvalidValue;
    if (!(MN ? encode(&map, w, 2, C, q.r, q.L, up16(q.r), true) : encode(&map, w, 2, q.r, C, q.L, Cfg::TN, true))) return cudaErrorInvalidValue;
    const int64_t tiles = row_tiles(q), sms = device_info().num_sms;
    const int64_t G = sms / tiles < 1 ? 1 : sms / tiles;
    const cudaError_t e = ensure_dynamic_smem((const void *)expand_kernel<Cfg>, Cfg::SMEM);
    if (e != cudaSuccess) return e;
    return launch_dependent(expand_kernel<Cfg>, dim3((unsigned)(tiles > sms ? tiles : sms)), E_THREADS, Cfg::SMEM, 1, s, rows, map, from, to, params(q, C), base, out, (int)sms,
                            (int)G);
}
template <bool MN>
static cudaError_t expand(const LoraPlan &q, const void *v, const void *w, int dtype, const void *base, void *out, int C, cudaStream_t s) {
    if (dtype == ZFFN_DT_BF16) return q.r <= 64 ? expand<2, 128, 1, MN>(q, v, w, base, out, C, s) : expand<2, 128, 2, MN>(q, v, w, base, out, C, s);
    return q.r <= 64 ? expand<4, 128, 1, MN>(q, v, w, base, out, C, s) : expand<4, 64, 2, MN>(q, v, w, base, out, C, s);
}

static bool outer_job(OuterJob *job, const LoraPlan &q, const void *v16, const void *x, void *d, int C, bool transposed) {
    *job = OuterJob{};
    job->x = static_cast<const __nv_bfloat16 *>(x);
    job->v16 = static_cast<const __nv_bfloat16 *>(v16);
    job->d = d;
    job->C = C;
    job->n_tiles = (C + 127) / 128;
    job->wide_x = C % 64 == 0;
    job->transposed = transposed;
    return encode(&job->xm, x, 2, C, q.T, 1, KB, false, job->wide_x ? 2 : 0) &&
           encode(&job->vm, v16, 2, pieces_pitch(q.r), q.T, 1, KB, false, pieces_pitch(q.r) / 64);
}
template <int BOXES>
static cudaError_t outer(const LoraPlan &q, const OuterJob &a, const OuterJob &b, int dtype, int part_log, cudaStream_t s) {
    using Cfg = OuterCfg<BOXES>;
    const int n_tiles = a.n_tiles + b.n_tiles;
    const int64_t tiles = (int64_t)q.L * n_tiles, sms = device_info().num_sms;
    if (tiles + sms > 0x7fffffff) return cudaErrorInvalidValue;
    Params p = params(q, 0);
    p.each = GroupWalk<128, 1, true>::divisor(n_tiles);
    const cudaError_t e = ensure_dynamic_smem((const void *)outer_kernel<Cfg>, Cfg::SMEM);
    if (e != cudaSuccess) return e;
    return launch_dependent(outer_kernel<Cfg>, dim3((unsigned)(tiles < sms ? tiles : sms)), O_THREADS, Cfg::SMEM, 1, s, a, b, p,
                            (int)(dtype == ZFFN_DT_BF16), part_log);
}

}  // namespace lora

size_t lora_pieces_bytes(int T, int r) { return (size_t)T * 2 * lora::pieces_pitch(r); }
bool lora_by_rows(int T, int r, int L) { return lora::few(T, r, L); }

cudaError_t launch_lora_shrink(const LoraPlan &q, const void *x, const void *w, bool transposed, float *v, void *v16, const float *other, void *other16,
                               int C, cudaStream_t s) {
    using namespace lora;
    if (!encode_fn()) return cudaErrorNotSupported;
    return transposed ? shrink<true>(q, x, w, v, v16, other, other16, C, s) : shrink<false>(q, x, w, v, v16, other, other16, C, s);
}

cudaError_t launch_lora_expand(const LoraPlan &q, const void *v16, const void *w, bool transposed, int dtype, const void *base, void *out, int C,
                               cudaStream_t s) {
    using namespace lora;
    if (!encode_fn()) return cudaErrorNotSupported;
    return transposed ? expand<true>(q, v16, w, dtype, base, out, C, s) : expand<false>(q, v16, w, dtype, base, out, C, s);
}

cudaError_t launch_lora_rows(const LoraPlan &q, const void *x, const void *A, const void *B, int dtype, const void *base, void *out, float *v, int N, int K,
                             cudaStream_t s) {
    using namespace lora;
    const __nv_bfloat16 *x16 = static_cast<const __nv_bfloat16 *>(x), *a16 = static_cast<const __nv_bfloat16 *>(A), *b16 = static_cast<const __nv_bfloat16 *>(B);
    const int64_t sms = device_info().num_sms;
    const dim3 rows((unsigned)q.T, (unsigned)(q.r / 8));
    const cudaError_t e = (int64_t)rows.x * rows.y <= 2 * sms ? launch_dependent(shrink_row_kernel<2>, rows, 512, 0, 1, s, params(q, K), x16, a16, v)
                                                         : launch_dependent(shrink_row_kernel<1>, rows, 256, 0, 1, s, params(q, K), x16, a16, v);
    if (e != cudaSuccess) return e;
    auto expand = [&](auto *to) {
        using O = std::remove_pointer_t<decltype(to)>;
        const O *from = static_cast<const O *>(base);
        if (lane_wide(q.r)) {
            const int g = q.r / 8;
            const int64_t chunks = ((int64_t)N * g + 8 * R_THREADS - 1) / (8 * R_THREADS), at_once = std::max<int64_t>(1, 12 * sms / q.T);
            const int64_t turns = (chunks + at_once - 1) / at_once;
            return launch_dependent(expand_lane_kernel<O>, dim3((unsigned)q.T, (unsigned)((chunks + turns - 1) / turns)), R_THREADS, 0, 1, s, params(q, N), v, b16, from, to, __builtin_ctz(g));
        }
        return launch_dependent(expand_row_kernel<O>, dim3((unsigned)q.T, (unsigned)((N + 2 * R_THREADS - 1) / (2 * R_THREADS))), R_THREADS, 0, 1, s, params(q, N), v, b16, from, to);
    };
    return dtype == ZFFN_DT_BF16 ? expand(static_cast<__nv_bfloat16 *>(out)) : expand(static_cast<float *>(out));
}

cudaError_t launch_lora_outer(const LoraPlan &q, const void *dv16, const void *x, void *dA, int K, const void *v16, const void *dy, void *dB, int N, int dtype,
                              cudaStream_t s) {
    using namespace lora;
    if (!encode_fn()) return cudaErrorNotSupported;
    OuterJob a, b;
    if (!outer_job(&a, q, dv16, x, dA, K, false) || !outer_job(&b, q, v16, dy, dB, N, true)) return cudaErrorInvalidValue;
    // (several parts: columns for their sum as well, so that one accumulator alone has room from r = 72)
    const bool one = 4 * up16(q.r) > 256;
    const int part_log = one && dtype == ZFFN_DT_BF16 ? LONG_PART_LOG : PART_LOG;
    const int boxes = one && q.T > KB << part_log ? 6 : pieces_pitch(q.r) / 64;
    return boxes <= 2 ? outer<2>(q, a, b, dtype, part_log, s) : boxes <= 4 ? outer<4>(q, a, b, dtype, part_log, s) : outer<6>(q, a, b, dtype, part_log, s);
}

}  // namespace zffn
