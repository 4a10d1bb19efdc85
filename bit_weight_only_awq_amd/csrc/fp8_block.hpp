// fp8_block.hpp -- E4M3 codes with a scale for each block of 128, shared by the
// quantiser (fp8_block.hip), the streaming product (stream_fp8_block.hip) and
// the LDS-pipelined one (gemm_fp8_block.hip).
//
// y[m,n] = sum over blocks b of 128 along K of sa[m][b] sw[n / 128][b] t, with
// t = sum_{k in b} a[m][k] w[n][k] of one v_mfma_scale_f32_16x16x128_f8f6f4 with unit
// scales: the instruction's 128 k are one block, so a block's sum leaves the
// matrix cores once, in fp32, and is added to the running sums by one FMA a
// value.  (The instruction's own scales are powers of two and cannot take
// these.)  The weights are the A operand and the tokens the B operand: a
// lane then holds four consecutive outputs n of one token, and its token's scale
// is one register.
//
// Both matrices are K-major, so an operand is 32 bytes of one row a lane.  Which 32 of
// the 128 is free as long as both operands agree: lane group gq = lane / 16 takes
// bytes 16 gq .. + 15 of either half of the block, so that a load of 16 bytes a lane covers
// 64 consecutive bytes of 16 rows.
#pragma once

#include "device.hpp"
#include "fp8_ops.hpp"
#include "launch.hpp"
#include "moe.hpp"

namespace awq4 {

constexpr int kBlk = 128;              // values of a block
constexpr uint32_t kOut = 0x80000000u;  // offset past every buffer (each under 2^31 bytes): loads read zero

__device__ __forceinline__ i32x8 operand32(u32x4 lo, u32x4 hi) {
    return (i32x8){(int32_t)lo[0], (int32_t)lo[1], (int32_t)lo[2], (int32_t)lo[3],
                   (int32_t)hi[0], (int32_t)hi[1], (int32_t)hi[2], (int32_t)hi[3]};
}

// One tile: its rows and the matrices it reads.
struct Fp8Tile {
    const uint8_t *a, *w;    // a: row row0, or row 0 where rows are gathered
    const float *sa, *sw;
    int tile_n, row0, rows;  // rows: those of the tile that exist
    int a_rows;              // rows that `a` may be read for
    bool gather;
};
__device__ __forceinline__ Fp8Tile fp8_tile(const Fp8BlockArgs &g, const GroupTile &q, int BM) {
    Fp8Tile t;
    const int blocks = (g.K + kBlk - 1) / kBlk;
    t.gather = g.groups.rows != nullptr;
    t.tile_n = q.tile_n;
    t.row0 = q.row0;
    t.rows = min(q.row_end - q.row0, BM);
    t.a_rows = t.gather ? g.groups.x_rows : t.rows;
    const size_t first = t.gather ? 0 : (size_t)t.row0, e = q.expert;
    t.a = g.a + first * g.K;
    t.sa = g.sa + first * blocks;
    t.w = g.w + e * (size_t)g.N * g.K;
    t.sw = g.sw + e * (size_t)((g.N + kBlk - 1) / kBlk) * blocks;
    return t;
}
// Row of t.a that the tile's row r reads, or -1 where the tile has no such row.
__device__ __forceinline__ int fp8_source(const Fp8BlockArgs &g, const Fp8Tile &t, int r) {
    if (r >= t.rows) return -1;
    return t.gather ? group_source(g.groups.rows, t.row0 + r, g.groups.top, g.groups.x_rows) : r;
}

}  // namespace awq4
