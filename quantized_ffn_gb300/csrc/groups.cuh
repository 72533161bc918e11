// groups.cuh -- a warp's walk over the tiles of rows that are grouped by expert or
// adapter.
#pragma once

#include "zffn_internal.cuh"

namespace zffn {

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
    bool rest;                   // tiles of the rows of none as well
    int t;                       // the tile that get() gives
    int e0, before, top;         // groups held from e0 on; row tiles and largest offset before them
    int lo, hi, n, inc;          // the lane's group: rows, row tiles, and those up to it
    // what get() gives: rows row0 .. row0 + rows - 1 of group e, tile nt of the other matrix
    int e, row0, rows, nt;

    __device__ __forceinline__ void start(const int32_t *offsets_, int M_, int E_, int n_tiles_, bool rest_, int first) {
        offsets = offsets_; M = M_; E = E_; n_tiles = n_tiles_; rest = rest_; t = first;
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
        if (WHOLE) n = g < E;
        inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
    }
    // Tile t; false past the last one.
    __device__ __forceinline__ bool get() {
        for (;;) {
            const unsigned past = __ballot_sync(0xffffffffu, t < (before + inc) * n_tiles);
            if (past) {
                const int l = __ffs(past) - 1;
                const int first = __shfl_sync(0xffffffffu, inc - n, l), tiles = __shfl_sync(0xffffffffu, n, l);
                const int at = __shfl_sync(0xffffffffu, lo, l), end = __shfl_sync(0xffffffffu, hi, l);
                e = e0 + l;
                int in = t - (before + first) * n_tiles;
                const int block = in / (GROUP * n_tiles) * GROUP, wide = min(GROUP, tiles - block);
                in -= block * n_tiles;
                nt = in / wide;
                row0 = at + (WHOLE ? 0 : (block + in - nt * wide) * TM);
                rows = WHOLE ? end - at : min(TM, end - row0);
                return true;
            }
            before += __shfl_sync(0xffffffffu, inc, 31);
            if (e0 + 32 > E) return false;
            hold(e0 + 32);
        }
    }
};

}  // namespace zffn
