// moe.hpp -- products grouped by expert: which tile of which expert a workgroup takes.
//
// The rows of a grouped product lie in the order of their experts, expert e's
// from offsets[e] to offsets[e + 1] - 1; how many each has is known on the
// device only.  A launch has as many workgroups as any split of its rows over
// the experts can need (the host's bound), each finds its tile from the offsets
// by itself, and those past the last tile end at once: no tile list in memory,
// no launch of its own to make one, nothing for the host to wait for.
#pragma once

#include "device.hpp"
#include "launch.hpp"

namespace awq4 {

struct GroupTile {
    int expert;
    int tile_n;         // column tile
    int row0, row_end;  // its rows: row0 .. min(row0 + BM, row_end) - 1
    int index;          // number of the tile, below the launch's bound on them
    bool live;
};

// Offsets outside 0 .. R are taken as the nearest of the two, and an expert whose rows would end
// before they begin has none: whatever the offsets hold, every row is below R.
__device__ __forceinline__ int group_offset(const int32_t *__restrict__ offsets, int e, int R) {
    return min(max(offsets[e], 0), R);
}

// Tile of workgroup i: BM rows of an expert and one of tiles_n column tiles; at most max_tiles tiles
// of rows.  Every wave computes it for itself: a lane counts the tiles of ceil(E / 64) consecutive
// experts, a scan over the lanes gives where they begin.  The tiles of an expert lie
// together, its row tiles fastest, so that the workgroups of one die read the same weights at the same time.
__device__ __forceinline__ GroupTile group_tile(const int32_t *__restrict__ offsets, int E, int R, int BM, int tiles_n,
                                                int max_tiles, int i) {
    const int lane = threadIdx.x & 63;
    const int per = (E + 63) >> 6;
    const int e0 = lane * per, e1 = min(E, e0 + per);
    int n = 0;
    if (e0 < e1) {
        int lo = group_offset(offsets, e0, R);
        for (int e = e0; e < e1; ++e) {
            const int hi = group_offset(offsets, e + 1, R);
            n += (max(hi - lo, 0) + BM - 1) / BM;
            lo = hi;
        }
    }
    int end = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(end, d, 64);
        if (lane >= d) end += v;
    }
    GroupTile t;
    const int total = min(__builtin_amdgcn_readlane(end, 63), max_tiles) * tiles_n;
    t.live = i < total;
    if (!t.live) return t;
    const int id = tile_of_xcd_order(i, total);
    const int row_tile = id / tiles_n;
    const int owner = __builtin_ctzll(__ballot(end > row_tile));
    int first = __builtin_amdgcn_readlane(end - n, owner);
    int e = owner * per, count = 0, lo = 0, hi = 0;
    for (;; ++e) {
        lo = __builtin_amdgcn_readfirstlane(group_offset(offsets, e, R));
        hi = __builtin_amdgcn_readfirstlane(group_offset(offsets, e + 1, R));
        count = (max(hi - lo, 0) + BM - 1) / BM;
        if (first + count > row_tile || e + 1 >= E) break;
        first += count;
    }
    const int local = id - first * tiles_n;
    t.expert = e;
    t.tile_n = local / count;
    t.row0 = lo + (local - t.tile_n * count) * BM;
    t.row_end = hi;
    t.index = id;
    return t;
}

// Row of x that row r of the product reads: slot rows[r] of the (token, place) slots, `top` to a
// token.  A slot that names no row of x reads row 0.
__device__ __forceinline__ int group_source(const int32_t *__restrict__ rows, int r, int top, int x_rows) {
    const int s = rows[r];
    const int t = s / top;
    return s >= 0 && t < x_rows ? t : 0;
}

}  // namespace awq4
