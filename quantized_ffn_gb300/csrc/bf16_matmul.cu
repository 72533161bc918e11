// bf16_matmul.cu -- products of bf16 matrices on the 5th-generation tensor cores, dense
// or grouped by expert, and their gradients:
//     forward    y[m][n]     = sum_k a[m][k] w[e][n][k]
//     back       y[m][n]     = sum_k a[m][k] w[e][k][n]
//     weights    dw[e][n][k] = sum_m dy[m][n] a[m][k]      over expert e's rows m
// Sums are fp32, in tensor memory, over the contraction or (long ones) parts of it that are
// joined in fp32, and are rounded once.
// An operand whose contracted index runs along its rows' memory is taken K-major, the
// other ones (w in `back`, both in `weights`) as they lie in memory, MN-major: nothing
// is transposed on the way.
#include <atomic>

#include "bf16.h"
#include "groups.cuh"
#include "launch.cuh"
#include "roles.cuh"
#include "tiles.cuh"

namespace zffn {
namespace b16 {

enum Kind { FORWARD, BACK, WEIGHTS };

// Stages of a part, as a logarithm.  The tensor core's adds drop what is below the accumulator's
// last bit, so that a long sum comes out short (of positive values, even in [0.5, 1.5]: of 512 2.3e-7, of 2048
// 2.3e-6, of 4096 7.9e-6, of 32768 1.5e-4, of 65536 some 3e-4).  Parts of 512, joined in fp32 registers that
// round to nearest, hold it at 2.3e-7 whatever the length (up to 65536 values no more than 9e-7 of any
// sum).  Also of a bf16 result: of sums of 2048 products 1 in 800 was not the nearest bf16 value in
// one part, 1 in 2600 is in four, as of fp32 sums by the ordinary units (32768 rows of 128 experts,
// 1536 x 2048: 198 / 204 us, 2048 rows of 128 and one token's experts the same).
constexpr int PART_LOG = 3;

struct Params {
    const int32_t *offsets;
    void *y;
    int *err;
    int M, N, K, E;
    int n_tiles;        // tiles of w's rows; weights: of dw[e]'s columns
    int m_tiles;        // weights: tiles of dw[e]'s rows
    int y_bf16;
    int vec;            // y's rows are 16-byte multiples
    // an MN-major operand whose rows are whole boxes wide (the columns a multiple of 64):
    // one copy takes all boxes of a tile, its map counting boxes by an index of their own.
    // (With a copy a box the one issuing thread held the weights' gradients back: an even
    // 256 rows of 128 experts, 1536 x 2048, 185 us against 202.)
    int wide_a, wide_w;
    FastDiv each, across;   // of the walk; weights: by n_tiles
};
// a: forward, back: [M][K]; weights: dy, in boxes of 16, 32 and 64 rows.  w: w; weights: a,
// in the same.  y: what the stores go to.
struct Maps {
    CUtensorMap a[3], w[3], y;
};

// ---------------------------------------------------------------------------
// Many rows: tiles of 128 rows (a CTA pair: 256) times 256 columns of the result, a
// (weights: dy) on the MMA's M side.  Persistent: every cluster takes tiles in turn;
// two accumulators in tensor memory, so that one is taken out while the next tile's
// MMAs run.  PARTS: a long sum in parts (see PART_LOG), joined in the registers of the
// threads that take them out.
//
// Roles: warps 0 .. 7 take a tile out of tensor memory (32 rows by 128 columns each) and
// write it, warp 8 loads by TMA, warp 9 issues the MMAs; weights: warp 10 zeroes the rows past an
// expert's last in its last stage (in the MMA's own warp that held the MMAs back: 32768
// rows of 128 experts, 1536 x 2048, 217 us).  Those 32768 rows, unevenly, ten calls on the same
// inputs: forward 205 us, 1.01 PFLOP/s, on tiles that end with an expert's rows (49,400 rows of
// MMAs); weights 202 us, 1.02 PFLOP/s, bound by the way from L2 (four stages a tile, and then it is
// written).  In a loop of seconds over changing inputs, at the power limit, 229 and 210.
// ---------------------------------------------------------------------------
template <int KIND_, bool PAIR_, bool PARTS_>
struct LargeCfg {
    static constexpr int KIND = KIND_;
    static constexpr bool PAIR = PAIR_, PARTS = PARTS_;
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int TM = 128 * CTAS, TN = 256;
    static constexpr bool A_MN = KIND == WEIGHTS, W_MN = KIND != FORWARD;
    static constexpr int W_ROWS = TN / CTAS;                 // of the tile's columns that a CTA holds
    static constexpr int A_BYTES = 128 * 128;
    static constexpr int STAGE = A_BYTES + W_ROWS * 128;
    static constexpr int NS = PAIR ? 6 : 4;
    static constexpr int EPI = 8;
    static constexpr int THREADS = (EPI + 2 + (KIND == WEIGHTS)) * 32;
    static constexpr int OUT_BYTES = 4096;                   // a warp's box of 32 rows x 128 bytes
    static constexpr int OFF_OUT = NS * STAGE;
    static constexpr int OFF_BAR = OFF_OUT + EPI * OUT_BYTES;
    static constexpr int SMEM = OFF_BAR + (3 * NS + 5) * 8 + 16 + 1024;
    using Walk = GroupWalk<TM, 8, KIND == WEIGHTS>;
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) large_kernel(const __grid_constant__ Maps maps, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *s_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *s_empty = s_full + C::NS, *t_full = s_empty + C::NS, *t_empty = t_full + 2, *done = t_empty + 2;
    uint64_t *cut_full = done + 1;                           // weights: an expert's last rows
    int *info = reinterpret_cast<int *>(cut_full + C::NS);   // abort, TMEM base, stages that the loads have begun
    volatile int *abort_flag = info, *begun = info + 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = C::PAIR ? (int)cluster_ctarank() : 0;
    constexpr bool GRAD = C::KIND == WEIGHTS;

    if (warp == C::EPI && lane == 0) {
        info[0] = info[2] = 0;
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(&s_full[i], GRAD && C::PAIR ? 2 : 1);
            mbar_init(&s_empty[i], 1);
            mbar_init(&cut_full[i], 1);
        }
        for (int i = 0; i < 2; ++i) { mbar_init(&t_full[i], 1); mbar_init(&t_empty[i], C::EPI * C::CTAS); }
        mbar_init(done, 1);
        fence_mbarrier_init();
        for (int i = 0; i < (GRAD ? 3 : 1); ++i) {
            prefetch_tensormap(&maps.a[i]);
            prefetch_tensormap(&maps.w[i]);
        }
    }
    if (warp == C::EPI + 1) {
        uint32_t *dst = reinterpret_cast<uint32_t *>(info + 1);
        if constexpr (C::PAIR) { tmem_alloc_pair(dst, 512); tmem_relinquish_pair(); }
        else { tmem_alloc(dst, 512); tmem_relinquish(); }
        tc_fence_before();
    }
    __syncthreads();
    grid_wait();
    grid_launch_dependents();          // (this block has its tensor memory)
    if (C::PAIR) cluster_sync_all();   // the peer's barriers are set up
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(info + 1);
    typename C::Walk wk;
    wk.start(p.offsets, p.M, p.E, GRAD ? p.m_tiles * p.n_tiles : p.n_tiles, p.each, !GRAD, blockIdx.x / C::CTAS);
    const int step = gridDim.x / C::CTAS;
    constexpr int part_log = C::PARTS ? PART_LOG : 30, part_mask = (1 << part_log) - 1;
    // stages of the tile at hand (none: zeros)
    auto blocks = [&] { return GRAD ? (wk.rows + KB - 1) / KB : wk.e < p.E ? (p.K + KB - 1) / KB : 0; };
    // groups of 16 contracted values in stage i
    auto steps = [&](int i) { return (min(KB, (GRAD ? wk.rows : p.K) - i * KB) + 15) / 16; };

    // weights: which boxes (16, 32 or 64 rows) hold that many groups of 16
    auto box_of = [](int n) { return n > 2 ? 2 : n - 1; };

    // Weights: rows of the next expert among a stage's last 16 become zeros, in both operands
    // (whatever they hold may be infinite).  A warp, after the copies and before the MMAs.
    auto zero_past = [&](uint32_t sa, uint32_t sw, int valid, int n) {
        if (valid >= n * 16) return;
        const uint32_t box = 2048u << box_of(n);
        const int each = (n * 16 - valid) * 8;               // chunks of 16 bytes in a box
        for (int c = lane; c < each; c += 32)
#pragma unroll
            for (int b = 0; b < 2 + C::W_ROWS / 64; ++b)
                st_shared_v4((b < 2 ? sa + b * box : sw + (b - 2) * box) + valid * 128 + c * 16, 0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
    };

    if (warp == C::EPI) {
        // ---- TMA producer
        const uint32_t full0 = C::PAIR ? mapa_shared(smem_u32(s_full), 0) : 0;
        uint32_t it = 0, cut_used = 0, cut_phase = 0;         // cut_full: stages that used it, each one's last phase
        bool ok = true;
        for (; ok && wk.get(); wk.t += step) {
            const int nb = blocks();
            const int mt = GRAD ? p.across.div(wk.nt) : 0, nt = GRAD ? wk.nt - mt * p.n_tiles : wk.nt;
            for (int i = 0; i < nb && lane == 0; ++i, ++it) {
                const uint32_t s = it % C::NS;
                if (it >= C::NS && !bar_wait(&s_empty[s], ((it / C::NS) & 1) ^ 1, abort_flag, p.err)) { ok = false; break; }
                uint8_t *sa = smem + s * C::STAGE, *sw = sa + C::A_BYTES;
                if constexpr (GRAD) {
                    *begun = (int)it;
                    // (of an expert's last rows no more than the MMA takes, or half as many again)
                    const int row = wk.row0 + i * KB, x = box_of(steps(i)), bytes = 2048 << x;
                    constexpr int WB = C::W_ROWS / 64;
                    const int c0 = mt * C::TM + rank * 128, c1 = nt * C::TN + rank * C::W_ROWS;
                    // s_full counts an arrival of each CTA.  Where rows have to be zeroed, the
                    // copies complete on a barrier of their own, and the arrival follows the
                    // zeroing.
                    const bool cut = wk.rows - i * KB < steps(i) * 16;
                    if (cut) {
                        mbar_arrive_expect_tx(&cut_full[s], (2 + WB) * bytes);
                        cut_phase ^= cut_used & (1u << s);
                        cut_used |= 1u << s;
                    }
                    if constexpr (C::PAIR) {
                        const uint32_t bar = cut ? smem_u32(&cut_full[s]) : full0 + s * 8;
                        if (!cut && rank == 0) mbar_arrive_expect_tx(&s_full[s], 2 * (2 + WB) * bytes);
                        else if (!cut) mbar_arrive_cluster(full0 + s * 8);
                        if (p.wide_a) tma_load_3d_pair(sa, &maps.a[x], bar, 0, row, c0 / 64);
                        else
                            for (int b = 0; b < 2; ++b) tma_load_2d_pair(sa + b * bytes, &maps.a[x], bar, c0 + b * 64, row);
                        if (p.wide_w) tma_load_3d_pair(sw, &maps.w[x], bar, 0, row, c1 / 64);
                        else
                            for (int b = 0; b < WB; ++b) tma_load_2d_pair(sw + b * bytes, &maps.w[x], bar, c1 + b * 64, row);
                    } else {
                        uint64_t *bar = cut ? &cut_full[s] : &s_full[s];
                        if (!cut) mbar_arrive_expect_tx(bar, (2 + WB) * bytes);
                        if (p.wide_a) tma_load_3d(sa, &maps.a[x], bar, 0, row, c0 / 64);
                        else
                            for (int b = 0; b < 2; ++b) tma_load_2d(sa + b * bytes, &maps.a[x], bar, c0 + b * 64, row);
                        if (p.wide_w) tma_load_3d(sw, &maps.w[x], bar, 0, row, c1 / 64);
                        else
                            for (int b = 0; b < WB; ++b) tma_load_2d(sw + b * bytes, &maps.w[x], bar, c1 + b * 64, row);
                    }
                } else {
                    if (rank == 0) mbar_arrive_expect_tx(&s_full[s], C::STAGE * C::CTAS);
                    const int col = wk.nt * C::TN + rank * C::W_ROWS;
                    if constexpr (C::PAIR) tma_load_2d_pair(sa, maps.a, full0 + s * 8, i * KB, wk.row0 + 128 * rank);
                    else tma_load_2d(sa, maps.a, &s_full[s], i * KB, wk.row0);
                    if constexpr (C::KIND == FORWARD) {
                        if constexpr (C::PAIR) tma_load_3d_pair(sw, maps.w, full0 + s * 8, i * KB, col, wk.e);
                        else tma_load_3d(sw, maps.w, &s_full[s], i * KB, col, wk.e);
                    } else if (p.wide_w) {
                        if constexpr (C::PAIR) tma_load_4d_pair(sw, maps.w, full0 + s * 8, 0, i * KB, col / 64, wk.e);
                        else tma_load_4d(sw, maps.w, &s_full[s], 0, i * KB, col / 64, wk.e);
                    } else {
                        for (int b = 0; b < C::W_ROWS / 64; ++b) {
                            if constexpr (C::PAIR) tma_load_3d_pair(sw + b * 8192, maps.w, full0 + s * 8, col + b * 64, i * KB, wk.e);
                            else tma_load_3d(sw + b * 8192, maps.w, &s_full[s], col + b * 64, i * KB, wk.e);
                        }
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok && !*abort_flag, 0);
        }
        // (a launch that gave up: wait for the copies in flight before leaving)
        if (lane == 0 && *abort_flag)
            for (uint32_t s = 0; s < C::NS; ++s)
                if ((cut_used >> s) & 1) mbar_wait(&cut_full[s], (cut_phase >> s) & 1, nullptr, p.err);
        if (lane == 0 && *abort_flag && rank == 0)
            for (uint32_t j = it > C::NS ? it - C::NS : 0; j < it; ++j)
                mbar_wait(&s_full[j % C::NS], (j / C::NS) & 1, nullptr, p.err);
        __syncwarp();
    } else if (warp == C::EPI + 1) {
        // ---- MMA issuer (of a pair: its first CTA)
        constexpr uint32_t idesc = idesc_bf16_f32(C::TM, C::TN, C::A_MN, C::W_MN);
        if (rank == 0) {
            uint32_t it = 0, acc = 0;
            bool ok = true;
            for (; ok && wk.get(); wk.t += step) {
                const int nb = blocks();
                if (nb == 0) continue;
                for (int i = 0; i < nb; ++i, ++it) {
                    const uint32_t s = it % C::NS, b = acc & 1, dst = tmem + b * 256;
                    const int at = i & part_mask;            // a part's first stage: 0
                    const bool last = at == part_mask || i == nb - 1;
                    if (at == 0) ok = acc < 2 || bar_wait_warp(&t_empty[b], ((acc >> 1) & 1) ^ 1, abort_flag, p.err);
                    ok = ok && bar_wait_warp(&s_full[s], (it / C::NS) & 1, abort_flag, p.err);
                    if (!ok) break;
                    const uint32_t sa = smem_u32(smem) + s * C::STAGE, sw = sa + C::A_BYTES;
                    const int n = steps(i);
                    const uint32_t box = GRAD ? 2048u << box_of(n) : 8192u;
                    tc_fence_after();
                    const uint64_t ad = C::A_MN ? smem_desc_mn_sw128(sa, box) : smem_desc_k_sw128(sa);
                    const uint64_t wd = C::W_MN ? smem_desc_mn_sw128(sw, box) : smem_desc_k_sw128(sw);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < KB / 16; ++k) {
                            if (k >= n) break;
                            if constexpr (C::PAIR) tc_mma_bf16_pair(dst, ad + k * k_step(C::A_MN), wd + k * k_step(C::W_MN), idesc, (at | k) != 0);
                            else tc_mma_bf16(dst, ad + k * k_step(C::A_MN), wd + k * k_step(C::W_MN), idesc, (at | k) != 0);
                        }
                        if constexpr (C::PAIR) {
                            tc_commit_pair(&s_empty[s]);
                            if (last) tc_commit_pair(&t_full[b]);
                        } else {
                            tc_commit(&s_empty[s]);
                            if (last) tc_commit(&t_full[b]);
                        }
                    }
                    __syncwarp();
                    acc += last;
                }
                ok = __all_sync(0xffffffffu, ok && !*abort_flag);
            }
            if (elect_one()) {
                if constexpr (C::PAIR) tc_commit_pair(done);
                else tc_commit(done);
            }
            __syncwarp();
        }
    } else if (warp == C::EPI + 2) {
        // ---- weights: zeroes the rows past an expert's last
        const uint32_t full0 = C::PAIR ? mapa_shared(smem_u32(s_full), 0) : 0;
        uint32_t it = 0, phases = 0;
        for (bool ok = true; ok && wk.get(); wk.t += step) {
            const int nb = blocks();
            it += nb;
            const int n = nb ? steps(nb - 1) : 0, valid = wk.rows - (nb - 1) * KB;
            if (valid >= n * 16) continue;
            const uint32_t s = (it - 1) % C::NS;
            // (the next such stage may be seconds away: the bound counts from the last stage begun)
            for (int tries = 0, at = *begun; !bar_test(&cut_full[s], (phases >> s) & 1); ++tries) {
                if (tries > (1 << 26)) {
                    const int now = *begun;
                    if (now == at) record_error(p.err, ZFFN_ERR_TIMEOUT), *abort_flag = 1;
                    tries = 0, at = now;
                }
                if ((tries & 1023) == 1023 && *abort_flag) { ok = false; break; }
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            phases ^= 1u << s;
            const uint32_t sa = smem_u32(smem) + s * C::STAGE;
            zero_past(sa, sa + C::A_BYTES, valid, n);
            if (lane == 0) {
                if constexpr (C::PAIR) mbar_arrive_cluster(full0 + s * 8);
                else mbar_arrive(&s_full[s]);
            }
            __syncwarp();
        }
    } else {
        // ---- take out and write: thread = one row of the tile
        const int q = warp & 3, half = warp >> 2;
        const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + half * 128;
        const uint32_t empty0 = C::PAIR ? mapa_shared(smem_u32(t_empty), 0) : 0;
        uint8_t *out = smem + C::OFF_OUT + warp * C::OUT_BYTES;
        uint32_t acc = 0;
        for (bool ok = true; ok && wk.get(); wk.t += step) {
            const int parts = (blocks() + part_mask) >> part_log;
            const bool some = parts != 0;
            const int mt = GRAD ? p.across.div(wk.nt) : 0, nt = GRAD ? wk.nt - mt * p.n_tiles : wk.nt;
            const int wrow = (GRAD ? mt * C::TM : 0) + 128 * rank + q * 32;   // this warp's first row (of dw[e], of the tile)
            const int left = GRAD ? p.N - wrow : wk.rows - wrow;
            const int64_t row = GRAD ? wrow : wk.row0 + wrow;
            const int cols = GRAD ? p.K : p.N;
            // The tile leaves in boxes of 128 bytes a row: by TMA where all 32 rows are the tile's
            // and 16-byte multiples, else by the lanes, a row's bytes by neighbouring ones.
            const int col0 = nt * C::TN + half * 128;
            const int need = min(4, (cols - col0 + 31) / 32);   // groups of 32 columns that are the result's
            uint32_t b = 0, from = 0;
            auto full = [&] {                                // the next part's sums are there
                b = acc & 1, from = taddr + b * 256;
                ok = bar_wait_warp(&t_full[b], (acc >> 1) & 1, abort_flag, p.err);
                tc_fence_after();
                ++acc;
            };
            auto taken = [&] {                               // the accumulator has been read
                if (!some) return;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (C::PAIR) mbar_arrive_cluster(empty0 + b * 8);
                    else mbar_arrive(&t_empty[b]);
                }
            };
            auto at = [&](int r, int chunk) { return out + r * 128 + ((chunk ^ (r & 7)) << 4); };
            auto fetch = [&](int l, uint32_t (&to)[32]) {
                if (some) tmem_ld_32x32b_x32(from + l * 32, to);
                else
#pragma unroll
                    for (int j = 0; j < 32; ++j) to[j] = 0;
            };
            auto write = [&](auto elem_size) {
                constexpr int elem = decltype(elem_size)::value, per = 128 / elem, LOADS = per / 32;
                constexpr bool PARTS = C::PARTS;
                uint32_t d[PARTS ? 4 : 2][32];
                if constexpr (PARTS) {                       // all parts' sums, as they come
                    float sum[4][32];
#pragma unroll
                    for (int l = 0; l < 4; ++l)
#pragma unroll
                        for (int j = 0; j < 32; ++j) sum[l][j] = 0.f;
                    for (int i = 0; i < parts; ++i) {
                        full();
                        if (!ok) return;
#pragma unroll
                        for (int l = 0; l < 8; ++l) {
                            if (l >= 2 * need) break;
                            uint32_t v[16];
                            tmem_ld_32x32b_x16(from + l * 16, v);
                            tmem_ld_wait(v);
#pragma unroll
                            for (int j = 0; j < 16; ++j) sum[l / 2][l % 2 * 16 + j] += __uint_as_float(v[j]);
                        }
                        taken();
                    }
#pragma unroll
                    for (int l = 0; l < 4; ++l)
#pragma unroll
                        for (int j = 0; j < 32; ++j) d[l][j] = __float_as_uint(sum[l][j]);
                    if (need <= 0) return;
                } else {
                    if (some) full();
                    if (!ok) return;
                    if (need <= 0) {
                        taken();
                        return;
                    }
                    fetch(0, d[0]);
                }
#pragma unroll
                for (int l = 0; l < 4; ++l) {
                    if (l >= need) break;
                    uint32_t (&v)[32] = d[PARTS ? l : l & 1];
                    if constexpr (!PARTS) {
                        if (some) tmem_ld_wait(v);
                        if (l + 1 < need) fetch(l + 1, d[(l + 1) & 1]);
                        else taken();
                    }
                    if (l % LOADS == 0) {                    // (the store before has read the box)
                        if (lane == 0) bulk_wait_group_read<0>();
                        __syncwarp();
                    }
#pragma unroll
                    for (int j = 0; j < 8 / LOADS; ++j) {
                        uint4 u;
                        if constexpr (elem == 2) {
                            const uint32_t *f = v + j * 8;
                            u = make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
                        } else {
                            const uint32_t *f = v + j * 4;
                            u = make_uint4(f[0], f[1], f[2], f[3]);
                        }
                        *reinterpret_cast<uint4 *>(at(lane, l % LOADS * (8 / LOADS) + j)) = u;
                    }
                    if (l % LOADS != LOADS - 1 && l + 1 < need) continue;
                    const int col = col0 + l / LOADS * per;
                    if (GRAD || (p.vec && left >= 32)) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if (left > 0) {
                                if constexpr (GRAD) tma_store_3d(&maps.y, smem_u32(out), col, (int)row, wk.e);
                                else tma_store_2d(&maps.y, smem_u32(out), col, (int)row);
                            }
                            bulk_commit_group();
                        }
                        continue;
                    }
                    __syncwarp();
                    uint8_t *y = static_cast<uint8_t *>(p.y) + row * p.N * elem + (int64_t)col * elem;
                    const int64_t pitch = (int64_t)p.N * elem;
                    const int bytes = min(per, p.N - col) * elem;
                    if (p.vec) {
                        for (int i = lane; i < 32 * 8; i += 32)
                            if (i / 8 < left && i % 8 * 16 < bytes)
                                *reinterpret_cast<uint4 *>(y + i / 8 * pitch + i % 8 * 16) = *reinterpret_cast<const uint4 *>(at(i / 8, i % 8));
                    } else {
#pragma unroll
                        for (int k = 0; k < LOADS; ++k) {
                            const int c = (lane + 32 * k) * elem;
#pragma unroll 4
                            for (int r = 0; r < 32; ++r) {
                                const uint8_t *src = at(r, c >> 4) + (c & 15);
                                if (r >= left || c >= bytes) continue;
                                if constexpr (elem == 2) *reinterpret_cast<uint16_t *>(y + c + r * pitch) = *reinterpret_cast<const uint16_t *>(src);
                                else *reinterpret_cast<uint32_t *>(y + c + r * pitch) = *reinterpret_cast<const uint32_t *>(src);
                            }
                        }
                    }
                    __syncwarp();
                }
            };
            if (p.y_bf16) write(std::integral_constant<int, 2>{});
            else write(std::integral_constant<int, 4>{});
        }
        if (lane == 0) bulk_wait_group_all();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    // (no commit's arrival is left on its way; the wait is bounded, so it begins when the
    // sums have been taken out)
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

// ---------------------------------------------------------------------------
// Few rows an expert: the weights on the MMA's M side.  A tile is 128 columns of the
// result times TN rows of a; each cluster takes tiles in turn.  Where the tiles are
// fewer than the SMs a cluster's blocks split K: row j's sums go to the shared memory
// of rank j % split, which adds them in rank order, so that the result is the same
// every time.  Bound by HBM: every weight is read once (2048 rows of 128 experts, 1536 x 2048:
// 123 to 126 us, 6.6 TB/s; 8 rows of 8 experts 12.0 us on the same inputs again, of which the launch
// and the join are 4, 13.6 and 3.7 TB/s on changing ones).
//
// Roles: warps 0 .. 3 take a tile out of tensor memory (32 columns of the result each)
// and write it, warp 4 loads by TMA, warp 5 issues the MMAs.
// ---------------------------------------------------------------------------
template <int KIND_, int TN_>
struct SmallCfg {
    static constexpr int KIND = KIND_, TN = TN_;
    static constexpr bool W_MN = KIND == BACK;
    static constexpr int W_BYTES = 128 * 128;
    static constexpr int STAGE = W_BYTES + TN * 128;
    static constexpr int BLOCKS = 2;                         // blocks an SM
    static constexpr int NS = TN == 64 ? 3 : TN == 32 ? 4 : 5;
    static constexpr int EPI = 4;
    static constexpr int THREADS = (EPI + 2) * 32;
    static constexpr int MAX_SPLIT = 8;
    static constexpr int TMEM_COLS = 4 * TN;                 // two accumulators, the parts' sums before the last
    static constexpr int PART_ROWS = TN + MAX_SPLIT - 1;     // split * ceil(TN / split), at most
    static constexpr int OFF_PART = NS * STAGE;              // sums [rank][row / split][128]
    static constexpr int OFF_BAR = OFF_PART + PART_ROWS * 512;
    static constexpr int SMEM = OFF_BAR + (2 * NS + 5) * 8 + 8 + 1024;
    using Walk = GroupWalk<TN, 8>;
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::BLOCKS) small_kernel(const __grid_constant__ Maps maps, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float *part = reinterpret_cast<float *>(smem + C::OFF_PART);
    uint64_t *s_full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *s_empty = s_full + C::NS, *t_full = s_empty + C::NS, *t_empty = t_full + 2, *done = t_empty + 2;
    int *info = reinterpret_cast<int *>(done + 1);           // abort, TMEM base
    volatile int *abort_flag = info;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t split;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(split));
    const uint32_t rank = cluster_ctarank();
    if (split > 1) cluster_arrive();                         // (waited for before another's memory is written)
    if (warp == C::EPI && lane == 0) {
        info[0] = 0;
        for (int i = 0; i < C::NS; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&t_full[i], 1); mbar_init(&t_empty[i], C::EPI); }
        mbar_init(done, 1);
        fence_mbarrier_init();
        prefetch_tensormap(maps.a);
        prefetch_tensormap(maps.w);
    }
    if (warp == C::EPI + 1) {
        tmem_alloc(reinterpret_cast<uint32_t *>(info + 1), C::TMEM_COLS);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    grid_wait();
    grid_launch_dependents();          // (this block has its tensor memory)
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(info + 1);
    const int blocks = (p.K + KB - 1) / KB;
    const int kb0 = blocks * rank / split, nkb = blocks * (rank + 1) / split - kb0;   // this rank's share of K
    const int step = gridDim.x / split;
    constexpr int part_mask = (1 << PART_LOG) - 1;
    typename C::Walk wk;
    wk.start(p.offsets, p.M, p.E, p.n_tiles, p.each, true, blockIdx.x / split);
    const uint32_t slice = (C::TN + split - 1) / split;      // rows of a tile that a rank adds up
    const uint32_t inverse = (65536 + split - 1) / split;    // j * inverse >> 16 = j / split for j < 64
    // (split > 1: no more tiles than clusters, so each has one at most, and its walk ends there)
    auto next = [&] {
        wk.t += step;
        return split == 1 && wk.get();
    };
    bool some_tile = false;            // warps 0 .. 3, split > 1: sums were sent
    int last_row0 = 0, last_rows = 0, last_nt = 0;

    if (warp == C::EPI) {
        // ---- TMA producer
        uint32_t it = 0;
        bool ok = true;
        for (bool have = wk.get(); ok && have; have = next()) {
            for (int i = kb0; i < kb0 + nkb && lane == 0 && wk.e < p.E; ++i, ++it) {
                const uint32_t s = it % C::NS;
                if (it >= C::NS && !bar_wait(&s_empty[s], ((it / C::NS) & 1) ^ 1, abort_flag, p.err)) { ok = false; break; }
                uint8_t *sw = smem + s * C::STAGE;
                mbar_arrive_expect_tx(&s_full[s], C::STAGE);
                if constexpr (!C::W_MN) {
                    tma_load_3d(sw, maps.w, &s_full[s], i * KB, wk.nt * 128, wk.e);
                } else if (p.wide_w) {
                    tma_load_4d(sw, maps.w, &s_full[s], 0, i * KB, wk.nt * 2, wk.e);
                } else {
                    for (int b = 0; b < 2; ++b) tma_load_3d(sw + b * 8192, maps.w, &s_full[s], wk.nt * 128 + b * 64, i * KB, wk.e);
                }
                tma_load_2d(sw + C::W_BYTES, maps.a, &s_full[s], i * KB, wk.row0);
            }
            ok = __shfl_sync(0xffffffffu, ok && !*abort_flag, 0);
        }
        if (lane == 0 && *abort_flag)   // wait for the copies in flight before the block leaves
            for (uint32_t j = it > C::NS ? it - C::NS : 0; j < it; ++j)
                mbar_wait(&s_full[j % C::NS], (j / C::NS) & 1, nullptr, p.err);
        __syncwarp();
    } else if (warp == C::EPI + 1) {
        // ---- MMA issuer
        constexpr uint32_t idesc = idesc_bf16_f32(128, C::TN, C::W_MN, false);
        uint32_t it = 0, acc = 0;
        bool ok = true;
        for (bool have = wk.get(); ok && have; have = next()) {
            if (wk.e >= p.E || nkb == 0) continue;
            for (int i = 0; i < nkb; ++i, ++it) {
                const uint32_t s = it % C::NS, b = acc & 1, dst = tmem + b * C::TN;
                const int at = i & part_mask;                // a part's first stage: 0
                const bool last = at == part_mask || i == nkb - 1;
                if (at == 0) ok = acc < 2 || bar_wait_warp(&t_empty[b], ((acc >> 1) & 1) ^ 1, abort_flag, p.err);
                ok = ok && bar_wait_warp(&s_full[s], (it / C::NS) & 1, abort_flag, p.err);
                if (!ok) break;
                tc_fence_after();
                const uint32_t sw = smem_u32(smem) + s * C::STAGE;
                const int n = (min(KB, p.K - (kb0 + i) * KB) + 15) / 16;
                const uint64_t wd = C::W_MN ? smem_desc_mn_sw128(sw, 8192) : smem_desc_k_sw128(sw);
                const uint64_t ad = smem_desc_k_sw128(sw + C::W_BYTES);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < KB / 16; ++k) {
                        if (k >= n) break;
                        tc_mma_bf16(dst, wd + k * k_step(C::W_MN), ad + k * k_step(false), idesc, (at | k) != 0);
                    }
                    tc_commit(&s_empty[s]);
                    if (last) tc_commit(&t_full[b]);
                }
                __syncwarp();
                acc += last;
            }
            ok = __all_sync(0xffffffffu, ok && !*abort_flag);
        }
        if (elect_one()) tc_commit(done);
        __syncwarp();
    } else {
        // ---- take out and write: thread = one column of the result
        const uint32_t taddr = tmem + ((uint32_t)(warp * 32) << 16);
        const int tid = threadIdx.x;
        uint32_t acc = 0;
        bool ok = true;
        for (bool have = wk.get(); ok && have; have = next()) {
            const int parts = wk.e < p.E ? (nkb + part_mask) >> PART_LOG : 0;
            const int n = wk.nt * 128 + tid;
            constexpr int CH = 16;
            if (split > 1) {
                cluster_wait();                              // every block of the cluster runs
                some_tile = true;
                last_row0 = wk.row0; last_rows = wk.rows; last_nt = wk.nt;
            }
            const uint32_t to = smem_u32(part + rank * slice * 128) + tid * 4;
            uint32_t b = 0;
            auto full = [&] {                                // the next part's sums are there
                b = acc & 1;
                ok = bar_wait_warp(&t_full[b], (acc >> 1) & 1, abort_flag, p.err);
                tc_fence_after();
                ++acc;
            };
            auto taken = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&t_empty[b]);
            };
            // sums of this part, and (add) of those before
            auto fetch = [&](int c, bool add, uint32_t (&d)[CH]) {
                tmem_ld_32x32b_x16(taddr + b * C::TN + c, d);
                tmem_ld_wait(d);
                if (!add) return;
                uint32_t sum[CH];
                tmem_ld_32x32b_x16(taddr + 2 * C::TN + c, sum);
                tmem_ld_wait(sum);
#pragma unroll
                for (int j = 0; j < CH; ++j) d[j] = __float_as_uint(__uint_as_float(sum[j]) + __uint_as_float(d[j]));
            };
            // (the parts' sums in tensor memory: in registers they made the code long, one expert of 24
            // rows 7.5 / 9.3 us)
#pragma unroll 1
            for (int i = 1; i < parts; ++i) {
                full();
                if (!ok) break;
#pragma unroll 1
                for (int c = 0; c < C::TN; c += CH) {
                    if (c >= wk.rows) break;
                    uint32_t d[CH];
                    fetch(c, i > 1, d);
                    tmem_st_32x32b_x16(taddr + 2 * C::TN + c, d);
                }
                tmem_st_wait();
                taken();
            }
            if (ok && parts) full();
            if (!ok) break;
#pragma unroll 1
            for (int c = 0; c < C::TN; c += CH) {
                if (c >= wk.rows) break;
                uint32_t d[CH];
                if (parts) fetch(c, parts > 1, d);
                else
#pragma unroll
                    for (int j = 0; j < CH; ++j) d[j] = 0;
                if (split > 1) {
#pragma unroll
                    for (int j = 0; j < CH; ++j)
                        if (c + j < wk.rows) {
                            const uint32_t at = (c + j) * inverse >> 16;
                            st_cluster_f32(mapa_shared(to + at * 512, c + j - at * split), __uint_as_float(d[j]));
                        }
                } else if (n < p.N) {
                    const int64_t at = (int64_t)(wk.row0 + c) * p.N + n;
#pragma unroll
                    for (int j = 0; j < CH; ++j)
                        if (c + j < wk.rows) {
                            if (p.y_bf16) static_cast<__nv_bfloat16 *>(p.y)[at + (int64_t)j * p.N] = __float2bfloat16_rn(__uint_as_float(d[j]));
                            else static_cast<float *>(p.y)[at + (int64_t)j * p.N] = __uint_as_float(d[j]);
                        }
                }
            }
            if (parts) taken();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (split > 1) {
        if (!some_tile) cluster_wait();                      // (who has not met the first barrier above)
        cluster_sync_all();
        if (some_tile) {
            // the ranks' sums in rank order
            const int n = last_nt * 128 + threadIdx.x;
            for (int j = rank, i = 0; j < last_rows; j += split, ++i) {
                float v = part[i * 128 + threadIdx.x];
                for (uint32_t r = 1; r < split; ++r) v += part[(r * slice + i) * 128 + threadIdx.x];
                const int64_t at = (int64_t)(last_row0 + j) * p.N + n;
                if (n < p.N) {
                    if (p.y_bf16) static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(v);
                    else static_cast<float *>(p.y)[at] = v;
                }
            }
        }
    }
    if (warp == C::EPI + 1) {
        if (lane == 0) mbar_wait(done, 0, nullptr, p.err);
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// ---- host -------------------------------------------------------------------

// Row tiles of at most tr rows, at most: every expert may have one cut tile, and so may
// the rows of none.
static int64_t row_tiles_bound(int M, int E, const int32_t *offsets, int tr) {
    if (!offsets) return ((int64_t)M + tr - 1) / tr;
    return M / tr + (E + 1 < M ? E + 1 : M);
}

template <class C>
static cudaError_t run_large(const Maps &maps, const Params &p, int64_t tiles, cudaStream_t s) {
    const DeviceInfo &di = device_info();
    if (tiles + di.num_sms > 0x7fffffff) return cudaErrorInvalidValue;
    int64_t clusters = di.num_sms / C::CTAS;
    if (tiles < clusters) clusters = tiles;
    const cudaError_t e = ensure_dynamic_smem((const void *)large_kernel<C>, C::SMEM);
    if (e != cudaSuccess) return e;
    return launch_dependent(large_kernel<C>, dim3((unsigned)(clusters * C::CTAS)), C::THREADS, C::SMEM, C::CTAS, s, maps, p);
}

template <class C>
static cudaError_t launch_large(const Bf16Args &a, cudaStream_t s) {
    Maps maps{};
    Params p{a.offsets, a.y, a.err, a.M, a.N, a.K, a.E, (a.N + C::TN - 1) / C::TN, 0, a.y_dtype == ZFFN_DT_BF16, 0, 0, C::KIND == BACK && a.N % 64 == 0, {}, {}};
    p.each = C::Walk::divisor(p.n_tiles);
    const int elem = p.y_bf16 ? 2 : 4;
    p.vec = a.N * elem % 16 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
    if (!encode(maps.a, a.a, 2, a.K, a.M, 1, 128, false)) return cudaErrorInvalidValue;
    if (!(C::KIND == FORWARD ? encode(maps.w, a.w, 2, a.K, a.N, a.E, C::W_ROWS, true) : encode(maps.w, a.w, 2, a.N, a.K, a.E, KB, true, p.wide_w ? C::W_ROWS / 64 : 0)))
        return cudaErrorInvalidValue;
    if (p.vec && !encode(&maps.y, a.y, elem, a.N, a.M, 1, 32, false)) return cudaErrorInvalidValue;
    return run_large<C>(maps, p, row_tiles_bound(a.M, a.E, a.offsets, C::TM) * p.n_tiles, s);
}

// Ask once a device for the largest share of shared memory, so that C::BLOCKS blocks run
// on an SM.
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

// Clusters of `split` small-tile blocks that the current device runs at once with one block
// an SM (the query counts one whatever the shared memory; asked once for each device and
// split, and again where it failed).
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
            return 1;
        }
        k.store(n, std::memory_order_relaxed);
    }
    return n;
}

template <class C>
static cudaError_t launch_small(const Bf16Args &a, cudaStream_t s) {
    const DeviceInfo &di = device_info();
    Maps maps{};
    Params p{a.offsets, a.y, a.err, a.M, a.N, a.K, a.E, (a.N + 127) / 128, 0, a.y_dtype == ZFFN_DT_BF16, 0, 0, C::KIND == BACK && a.N % 64 == 0, {}, {}};
    p.each = C::Walk::divisor(p.n_tiles);
    if (!encode(maps.a, a.a, 2, a.K, a.M, 1, C::TN, false)) return cudaErrorInvalidValue;
    if (!(C::KIND == FORWARD ? encode(maps.w, a.w, 2, a.K, a.N, a.E, 128, true) : encode(maps.w, a.w, 2, a.N, a.K, a.E, KB, true, p.wide_w ? 2 : 0)))
        return cudaErrorInvalidValue;
    cudaError_t e = ensure_dynamic_smem((const void *)small_kernel<C>, C::SMEM);
    if (e == cudaSuccess) e = prefer_shared<C>();
    if (e != cudaSuccess) return e;
    // fewer tiles than blocks: split K so that the blocks fill the SMs, two stages each at
    // least, and all clusters run at once (a second wave costs more than the split gains)
    const int64_t tiles = row_tiles_bound(a.M, a.E, a.offsets, C::TN) * p.n_tiles, slots = (int64_t)di.num_sms * C::BLOCKS;
    if (tiles + slots > 0x7fffffff) return cudaErrorInvalidValue;
    const int most = (a.K + KB - 1) / KB / 2;
    int split = most < C::MAX_SPLIT ? most : C::MAX_SPLIT;
    if (split > slots / tiles) split = (int)(slots / tiles);
    while (split > 1 && (int64_t)clusters_at_once<C>(split) * C::BLOCKS < tiles) --split;
    if (split < 1) split = 1;
    const int64_t clusters = split > 1 || tiles < slots ? tiles : slots;
    return launch_dependent(small_kernel<C>, dim3((unsigned)(clusters * split)), C::THREADS, C::SMEM, (unsigned)split, s, maps, p);
}

template <int KIND, bool PARTS>
static cudaError_t launch_tiles(const Bf16Args &a, cudaStream_t s) {
    // CTA pairs where few of their 256 rows are past an expert's (single and pair: 128 experts
    // of 96 rows 142 / 154, of 192 rows 184 / 176, of 256 rows 207 / 195, 8 of 4096 rows 139 / 124)
    if (a.M / a.E >= 192) return launch_large<LargeCfg<KIND, true, PARTS>>(a, s);
    return launch_large<LargeCfg<KIND, false, PARTS>>(a, s);
}

template <int KIND>
static cudaError_t launch(const Bf16Args &a, cudaStream_t s) {
    // Rows an expert, and 128 x 256 tiles at least.  Small tiles: the least of 16, 32 rows
    // that takes an expert's rows (with some spread over their mean) at once, so that its
    // weights are read once; of 64 where the large ones are so few that splitting K gains more
    // (times of 1536 x 2048 in us, small and large, these with their sums in one part: 128 experts of 24 rows 138 / 140, of 48
    // rows 135 / 144, of 64 rows 148 / 144; one of 64 rows 9.5 / 15.4, of 256 rows 11.7 / 15.7,
    // of 512 rows 15.9 / 16.0).
    const int64_t mean = a.offsets ? ((int64_t)a.M * 3 / 2 + a.E - 1) / a.E : a.M;
    if (mean <= 16) return launch_small<SmallCfg<KIND, 16>>(a, s);
    if (mean <= 32) return launch_small<SmallCfg<KIND, 32>>(a, s);
    const int64_t most = (int64_t)a.M / 128 + (a.E < a.M ? a.E : a.M), tiles = most * ((a.N + 255) / 256);
    if (tiles <= device_info().num_sms / 6) return launch_small<SmallCfg<KIND, 64>>(a, s);
    if (a.K > KB << PART_LOG) return launch_tiles<KIND, true>(a, s);
    return launch_tiles<KIND, false>(a, s);
}

template <class C>
static cudaError_t launch_weights(const Bf16GradArgs &a, cudaStream_t s) {
    Maps maps{};
    Params p{a.offsets, a.dw, a.err, a.M, a.N, a.K, a.E, (a.K + C::TN - 1) / C::TN, (a.N + C::TM - 1) / C::TM, a.dw_dtype == ZFFN_DT_BF16, 1,
                   a.N % 64 == 0, a.K % 64 == 0, {}, FastDiv((a.K + C::TN - 1) / C::TN)};
    p.each = C::Walk::divisor(p.m_tiles * p.n_tiles);
    for (int x = 0; x < 3; ++x)
        if (!encode(&maps.a[x], a.dy, 2, a.N, a.M, 1, 16 << x, false, p.wide_a ? 2 : 0) ||
            !encode(&maps.w[x], a.a, 2, a.K, a.M, 1, 16 << x, false, p.wide_w ? C::W_ROWS / 64 : 0))
            return cudaErrorInvalidValue;
    if (!encode(&maps.y, a.dw, p.y_bf16 ? 2 : 4, a.K, a.N, a.E, 32, true)) return cudaErrorInvalidValue;
    return run_large<C>(maps, p, (int64_t)a.E * p.m_tiles * p.n_tiles, s);
}

}  // namespace b16

cudaError_t launch_bf16_matmul(const Bf16Args &a, cudaStream_t s) {
    if (!encode_fn()) return cudaErrorNotSupported;
    return a.transposed ? b16::launch<b16::BACK>(a, s) : b16::launch<b16::FORWARD>(a, s);
}

cudaError_t launch_bf16_grad_w(const Bf16GradArgs &a, cudaStream_t s) {
    using namespace b16;
    if (!encode_fn()) return cudaErrorNotSupported;
    // CTA pairs where their tiles are four rounds at least (dw of 2056 x 1032, single and pair:
    // 128 experts of 24 rows 122 / 115 us, of 256 rows 260 / 228, one of 64 rows 6.5 / 7.5)
    const int64_t tiles = (int64_t)a.E * ((a.N + 255) / 256) * ((a.K + 255) / 256);
    const bool pair = tiles >= 2 * (int64_t)device_info().num_sms;
    // Several parts where an expert may have as many rows (how many it has the host does not know). A
    // part's registers cost 1 to 3% (fp32 dw of 2048 x 1536, 128 experts of 128 rows 312 / 316 us; bf16,
    // of 256 rows 197 / 202): of bf16 where the experts have as many in the mean, or where a sum in
    // one part might come out more than 1.5e-4 short, a twenty-fifth of its rounding.
    const bool parts = a.M > KB << PART_LOG && (a.dw_dtype == ZFFN_DT_F32 || a.M / a.E > KB << PART_LOG || a.M > 1 << 15);
    if (parts) return pair ? launch_weights<LargeCfg<WEIGHTS, true, true>>(a, s) : launch_weights<LargeCfg<WEIGHTS, false, true>>(a, s);
    return pair ? launch_weights<LargeCfg<WEIGHTS, true, false>>(a, s) : launch_weights<LargeCfg<WEIGHTS, false, false>>(a, s);
}

}  // namespace zffn
