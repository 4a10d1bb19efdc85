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
};

// Offsets outside 0 .. R are taken as the nearest of the two, and an expert whose rows would end
// before they begin has none: whatever the offsets hold, every row is below R.
// Without offsets all rows are the one expert's: a dense product.
__device__ __forceinline__ int group_offset(const int32_t *__restrict__ offsets, int e, int R) {
    return offsets ? min(max(offsets[e], 0), R) : e > 0 ? R : 0;
}

// The tiles of a grouped product: BM rows of an expert and one of tiles_n column tiles each.  Every wave
// makes it for itself: a lane counts the row tiles of ceil(E / 64) consecutive experts, a
// scan over the lanes gives where they begin.  The tiles of an expert lie together, its row tiles
// fastest, so that neighbours, on one die, read the same weights at the same time.
struct GroupMap {
    const int32_t *offsets;
    int E, R, BM, tiles_n, per;
    int row_tiles;          // of all experts, at most the launch's bound
    int lo, hi, end, n;     // of this lane: rows of its (first) expert; row tiles up to its last expert, and of its own

    __device__ __forceinline__ GroupMap(const Groups &g, int BM_, int tiles_n_)
        : offsets(g.offsets), E(g.E), R(g.R), BM(BM_), tiles_n(tiles_n_), per((g.E + 63) >> 6) {
        const int lane = threadIdx.x & 63;
        const int e0 = lane * per, e1 = min(E, e0 + per);
        n = lo = hi = 0;
        if (e0 < e1) {
            lo = group_offset(offsets, e0, R);
            hi = group_offset(offsets, e0 + 1, R);
            n = count(lo, hi);
            for (int e = e0 + 1, at = hi; e < e1; ++e) {
                const int next = group_offset(offsets, e + 1, R);
                n += count(at, next);
                at = next;
            }
        }
        end = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(end, d, 64);
            if (lane >= d) end += v;
        }
        row_tiles = min(__builtin_amdgcn_readlane(end, 63), g.max_tiles);
    }
    __device__ __forceinline__ int count(int from, int to) const { return (max(to - from, 0) + BM - 1) / BM; }
    __device__ __forceinline__ int tiles() const { return row_tiles * tiles_n; }
    // tile id < tiles()
    __device__ __forceinline__ GroupTile at(int id) const {
        const int row_tile = __builtin_amdgcn_readfirstlane(id / tiles_n);
        const int owner = __builtin_ctzll(__ballot(end > row_tile));
        int first = __builtin_amdgcn_readlane(end - n, owner);
        int e = owner * per;
        int from = __builtin_amdgcn_readlane(lo, owner), to = __builtin_amdgcn_readlane(hi, owner);
        int c = __builtin_amdgcn_readfirstlane(count(from, to));
        while (first + c <= row_tile && e + 1 < E) {  // (only where a lane has several experts)
            first += c;
            ++e;
            to = __builtin_amdgcn_readfirstlane(group_offset(offsets, e + 1, R));
            from = __builtin_amdgcn_readfirstlane(group_offset(offsets, e, R));
            c = __builtin_amdgcn_readfirstlane(count(from, to));
        }
        const int local = id - first * tiles_n;
        GroupTile t;
        t.expert = e;
        t.tile_n = __builtin_amdgcn_readfirstlane(local / c);
        t.row0 = from + (local - t.tile_n * c) * BM;
        t.row_end = to;
        return t;
    }
};

// Row of x that row r of the product reads: slot rows[r] of the (token, place) slots, `top` to a
// token.  A slot that names no row of x reads row 0.
__device__ __forceinline__ int group_source(const int32_t *__restrict__ rows, int r, int top, int x_rows) {
    const int s = rows[r];
    const int t = s / top;
    return s >= 0 && t < x_rows ? t : 0;
}

}  // namespace awq4
