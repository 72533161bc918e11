// groups.cuh -- a warp's walk over the tiles of rows that are grouped by expert or
// adapter.
#pragma once

#include "zffn_internal.cuh"

namespace zffn {

// n / d for n < 2^31 by a multiplication (a division takes a warp some hundred clocks,
// several for each tile; n + the product's high half stay below 2^32).
struct FastDiv {
    uint32_t d, m, s;
    FastDiv() = default;
    explicit FastDiv(uint32_t div) : d(div), m(0), s(0) {
        while ((1ull << s) < d) ++s;
        m = (uint32_t)(((1ull << 32) * ((1ull << s) - d)) / d + 1);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int div(int n) const { return (int)((__umulhi(m, (uint32_t)n) + (uint32_t)n) >> s); }
#endif
};

// Groups 0 .. E - 1 are rows offsets[g] .. offsets[g + 1] - 1, and group E the rows of
// none.  Whatever the array holds, an offset counts as the largest of those up to it,
// kept within [0, M], so that the groups part the rows and the tiles are never more
// than the grid is sized by.  Without offsets group 0 holds all rows.
//
// Tiles are numbered group by group; within a group, GROUP row tiles take a tile of
// the other matrix in turn.  The lanes hold 32 groups at a time; `t` only grows.
// Every function is called by a full warp.  Offsets are read from L2: the grid
// before this one may have written them while this SM's L1 held older ones.
template <int TM, int GROUP, bool WHOLE = false>   // WHOLE: each group is one row tile, also an empty one
struct GroupWalk {
    const int32_t *offsets;
    int M, E, n_tiles;
    FastDiv each;                // GROUP * n_tiles (WHOLE: n_tiles)
    bool rest;                   // tiles of the rows of none as well
    int t;                       // the tile that get() gives
    int e0, before, top;         // groups held from e0 on; row tiles and largest offset before them
    int lo, hi, n, inc;          // the lane's group: rows, row tiles, and those up to it
    // what get() gives: rows row0 .. row0 + rows - 1 of group e, tile nt of the other matrix
    int e, row0, rows, nt;

    static FastDiv divisor(int n_tiles) { return FastDiv((uint32_t)n_tiles * (WHOLE ? 1 : GROUP)); }
    __device__ __forceinline__ void start(const int32_t *offsets_, int M_, int E_, int n_tiles_, const FastDiv &each_, bool rest_, int first) {
        offsets = offsets_; M = M_; E = E_; n_tiles = n_tiles_; each = each_; rest = rest_; t = first;
        before = 0;
        top = 0;
        hold(0);
    }
    __device__ __forceinline__ int offset(int g) const { return min(max(__ldcg(offsets + g), 0), M); }
    __device__ __forceinline__ void hold(int first) {
        const int lane = threadIdx.x & 31, g = first + lane;
        e0 = first;
        if (offsets) {
            int m = max(top, g <= E ? offset(g) : 0);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, m, o);
                if (lane >= o) m = max(m, v);
            }
            lo = m;
            hi = __shfl_down_sync(0xffffffffu, m, 1);
            if (lane == 31) hi = g < E ? max(m, offset(g + 1)) : m;
            if (g == E) hi = rest ? M : lo;
            top = __shfl_sync(0xffffffffu, m, 31);
        } else {
            lo = g == 0 ? 0 : M;
            hi = M;
        }
        n = g > E ? 0 : (hi - lo + TM - 1) / TM;
        inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
    }
    // Tile t; false past the last one.
    __device__ __forceinline__ bool get() {
        if constexpr (WHOLE) {
            e = each.div(t);
            if (e >= E) return false;
            nt = t - e * n_tiles;
            while (e >= e0 + 32) hold(e0 + 32);
            row0 = __shfl_sync(0xffffffffu, lo, e - e0);
            rows = __shfl_sync(0xffffffffu, hi, e - e0) - row0;
            return true;
        } else {
            for (;;) {
                const unsigned past = __ballot_sync(0xffffffffu, t < (before + inc) * n_tiles);
                if (past) {
                    const int l = __ffs(past) - 1;
                    const int first = __shfl_sync(0xffffffffu, inc - n, l), tiles = __shfl_sync(0xffffffffu, n, l);
                    const int at = __shfl_sync(0xffffffffu, lo, l), end = __shfl_sync(0xffffffffu, hi, l);
                    e = e0 + l;
                    int in = t - (before + first) * n_tiles;
                    const int block = each.div(in) * GROUP, wide = min(GROUP, tiles - block);
                    in -= block * n_tiles;
                    // in / wide: below 2^16, so that the product is off by less than the half that is added
                    nt = (int)(((float)in + 0.5f) * __frcp_rn((float)wide));
                    row0 = at + (block + in - nt * wide) * TM;
                    rows = min(TM, end - row0);
                    return true;
                }
                before += __shfl_sync(0xffffffffu, inc, 31);
                if (e0 + 32 > E) return false;
                hold(e0 + 32);
            }
        }
    }
};

}  // namespace zffn
