// stream_fp8_block.hip -- block-scaled E4M3 products of few rows (fp8_block.hpp has
// the arithmetic): the weights are read once, straight into registers.
//
// A workgroup has 32 outputs n and one tile of 16 tokens; its 4 waves take the
// blocks of 128 k in turn (with a K split: of the workgroup's share of them), two
// blocks' loads in flight, and their sums are added through LDS in wave order at
// the end, then over the K splits in split order (split_exchange.hpp).  Bound by
// memory: one token through 4096 x 14336 takes 16 to 18 us in a graph, of which 13 are what the
// same loads take alone and 4 what the smallest call does (64 outputs a workgroup
// 18.7, 16 of them 18.2, 8 waves 18.2), and 15.3 to 15.8 where calls follow each other on a stream; 8 through
// 4096 x 4096 9.5.  Where tiles of 128 x 128 through LDS give
// every CU work, those are level at one row and faster from about four
// on (api.cpp: plan_fp8_block).
#include "fp8_block.hpp"
#include "split_exchange.hpp"

namespace awq4 {

constexpr int kFp8StreamWaves = 4;

template <int NT>
struct Fp8Buf {
    u32x4 w[NT][2], a[2];
    float sa, sw;
};

template <int DT>
__global__ __launch_bounds__(64 * kFp8StreamWaves, 2) void fp8_block_stream(Fp8BlockArgs g, uint64_t *__restrict__ ws) {
    constexpr int WV = kFp8StreamWaves, COLS = kFp8StreamCols, NT = COLS / 16, ROWS = 16, PITCH = COLS + 4;
    __shared__ __attribute__((aligned(16))) float red[WV * ROWS * PITCH];
    const int lane = threadIdx.x & 63, j = lane & 15, gq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const GroupMap map(g.groups, ROWS, (g.N + COLS - 1) / COLS);
    if ((int)blockIdx.x >= map.tiles()) return;
    const int index = tile_of_xcd_order(blockIdx.x, map.tiles());
    const Fp8Tile t = fp8_tile(g, map.at(index), ROWS);
    const int K = g.K, N = g.N, blocks = (K + kBlk - 1) / kBlk;
    const int n0 = t.tile_n * COLS;
    // this workgroup's blocks [lo, hi) and this wave's share of them
    const int S = gridDim.y, per = (blocks + S - 1) / S;
    const int lo = blockIdx.y * per, hi = min(blocks, lo + per);
    const int n = hi - lo > wave ? (hi - lo - wave + WV - 1) / WV : 0;
    // rows past the matrix, and k past K, are past the buffer: they read as zero
    const __amdgpu_buffer_rsrc_t wr = buf_rsrc(t.w + (size_t)n0 * K, (int64_t)min(COLS, N - n0) * K);
    const __amdgpu_buffer_rsrc_t ar = buf_rsrc(t.a, (int64_t)t.a_rows * K);
    const __amdgpu_buffer_rsrc_t sr = buf_rsrc(t.sa, (int64_t)t.a_rows * blocks * 4);
    const float *const sw = t.sw + (size_t)(n0 / kBlk) * blocks;
    uint32_t wo[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) wo[i] = (uint32_t)((16 * i + j) * K);
    const int src = fp8_source(g, t, j);
    const uint32_t ao = src < 0 ? kOut : (uint32_t)src * (uint32_t)K;
    const uint32_t so = src < 0 ? kOut : (uint32_t)src * (uint32_t)blocks * 4u;
    auto issue = [&](Fp8Buf<NT> &b, int blk) {
        const int k = blk * kBlk + 16 * gq;
        const uint32_t k0 = k < K ? (uint32_t)k : kOut, k1 = k + 64 < K ? (uint32_t)(k + 64) : kOut;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            b.w[i][0] = __builtin_amdgcn_raw_buffer_load_b128(wr, wo[i] + k0, 0, 2);
            b.w[i][1] = __builtin_amdgcn_raw_buffer_load_b128(wr, wo[i] + k1, 0, 2);
        }
        // (one of the offsets, or both, may be past the buffer: their bit is set once)
        b.a[0] = __builtin_amdgcn_raw_buffer_load_b128(ar, (ao | k0) & kOut ? kOut : ao + k0, 0, 0);
        b.a[1] = __builtin_amdgcn_raw_buffer_load_b128(ar, (ao | k1) & kOut ? kOut : ao + k1, 0, 0);
        b.sa = bit_as<float>(__builtin_amdgcn_raw_buffer_load_b32(sr, so + 4u * blk, 0, 0));
        b.sw = sw[blk];
    };
    f32x4 acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
    auto compute = [&](const Fp8Buf<NT> &b) {
        const i32x8 a = operand32(b.a[0], b.a[1]);
        const float sc = b.sa * b.sw;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const f32x4 p = mfma_fp8(operand32(b.w[i][0], b.w[i][1]), a, (f32x4){0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][r] = __builtin_fmaf(p[r], sc, acc[i][r]);
        }
    };
    // keeps a buffer's loads where they are issued, a block ahead of their use
    auto fence = [] {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    auto block_of = [&](int i) { return lo + wave + i * WV; };
    Fp8Buf<NT> b0, b1;
    if (n > 0) issue(b0, block_of(0));
    if (n > 1) issue(b1, block_of(1));
    fence();
    int i = 0;
    for (; i + 3 < n; i += 2) {
        compute(b0);
        issue(b0, block_of(i + 2));
        fence();
        compute(b1);
        issue(b1, block_of(i + 3));
        fence();
    }
    if (i < n) compute(b0);
    if (i + 2 < n) {
        issue(b0, block_of(i + 2));
        fence();
    }
    if (i + 1 < n) compute(b1);
    if (i + 2 < n) compute(b0);

    // lane: outputs n0 + 16 i + 4 gq + r of token j
#pragma unroll
    for (int i = 0; i < NT; ++i) *(f32x4 *)(red + (wave * ROWS + j) * PITCH + 16 * i + 4 * gq) = acc[i];
    __syncthreads();
    const size_t at = (size_t)t.row0 * N;
    tile_store_or_exchange<64 * WV, DT, ROWS, COLS, PITCH, WV>(
        red, [](int c) { return c; }, (uint16_t *)g.y + at, (uint32_t *)ws + index,
        (char *)ws + split_counters_bytes(gridDim.x) + at * 4, (size_t)g.M * N * 4, t.rows, N, t.tile_n, S, 0);
}

hipError_t launch_fp8_block_stream(const Fp8BlockArgs &g, const Fp8BlockPlan &p, hipStream_t st) {
    if (p.splits > 1 && p.acc == nullptr) return hipErrorInvalidValue;
    const dim3 grid((unsigned)(p.tiles_n * p.tiles_m), (unsigned)p.splits), block(64 * kFp8StreamWaves);
    if (g.dtype == DT_BF16) hipLaunchKernelGGL(fp8_block_stream<DT_BF16>, grid, block, 0, st, g, p.acc);
    else hipLaunchKernelGGL(fp8_block_stream<DT_F16>, grid, block, 0, st, g, p.acc);
    return hipGetLastError();
}

}  // namespace awq4
