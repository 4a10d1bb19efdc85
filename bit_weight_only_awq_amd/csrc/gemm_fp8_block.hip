// gemm_fp8_block.hip -- block-scaled E4M3 products of many rows (fp8_block.hpp
// has the arithmetic): tiles through LDS.
//
// A workgroup has a tile of BN outputs n by BM tokens, a wave NT x MT tiles of 16 x 16 of them: 256 x 256 by
// 8 waves, where experts or the matrix have fewer rows 256 x 128 and then 128 x 128 by 8 waves as well, one workgroup a
// CU; and K split over workgroups where even these are few (an fp32 sum for each split,
// added in split order by a launch of its own, split_sum.hip).  The smaller a tile, the more slots: what is in flight sets
// the rate where memory does (96 rows, 4096 -> 14336, tiles of 128 x 128: 23.4 us with four slots, 25.7 by four waves with
// two slots and two workgroups a CU, 26.8 by these with three).  A stage is one block of 128 k: 128 bytes of each row of
// both matrices, copied straight into one of SLOTS LDS slots.
//
// One barrier a stage, and no wave waits for LDS behind it: a wave holds all NT weight
// operands of the stage and goes through its tokens 16 at a time, the
// operand of the next 16 being read meanwhile.  When the last 16 are in
// registers, nothing of the stage is left to read: the barrier stands there.
// Behind it the slot takes the copies of the stage SLOTS further (in flight for a whole stage, or two or
// three with more slots), and each weight operand is replaced by the next stage's as soon as its last
// matrix-core instruction is issued.  (With the barrier at the stage's end, where the first
// operands of all waves are read at once while the matrix cores wait: 1566
// TFLOP/s at 4096 x 14336 x 4096 against 1850.  Two groups of waves taking turns at the
// matrix cores: 1480 -- one wave a SIMD cannot keep them busy beside its own FMAs.)
// The copies are issued one beside each of the instructions behind the barrier (all at once:
// 1750).  The scales of four blocks are copied together, 16 bytes a row
// (each block's for itself, 256 rows in 256 cache lines: 6 % of the time).
//
// The matrix cores' sum of a tile is added to the running ones LAG instructions later.  The
// sum's FMAs take issue slots from the matrix cores: beside four FMAs an instruction of 32 cycles
// takes 42, which bounds the rate to 3650 TFLOP/s on this card; 2370 to 2400 are reached
// where the tiles are as many as the CUs and K is long (4096 x 4096 x 14336), the rest goes to
// the LDS (192 KB read and 64 KB written a stage, 2048 cycles of it).  With K = 4096 a tile has 32 stages, beside
// which its first copies and its stores count: 1980 in one round (4096 x 4096 x 4096), 2030 in four (N = 16384).
// N = 14336 is 896 tiles, 3.5 for each CU where the last half is waited for in full: 1940, 248 to 262 us.  (Three
// rounds of it, and the other columns by the smaller tiles in a launch behind: 257 -> 245 us in a graph, but 264 as
// before where calls follow each other on a stream.  One workgroup a CU going through its tiles without a
// pause, the next one's copies under way before the last one's stores: 295 -> 285 us by tiles of 256 x 128, but 257 ->
// 269 by the large ones, whose registers it overflows.)
// With few rows the copies bound: 777 tokens through 64 experts' 2048 x 2048 (top 8, 97 rows each; 268 MB of weights)
// take 80 us, the same copies without a product 75 or so, the weights' alone 53; tiles of 128 x 128, which read the
// tokens twice as often, 96; 256 x 128 with two slots 93 where three are 80.  Neither another order of the blocks
// in each tile nor non-temporal copies and stores change that.
#include "fp8_block.hpp"

namespace awq4 {

// 16-byte segment s of row r is stored at s ^ blk_swz(r): the 16 rows of an
// operand read lie on 16 different bank groups of 256 bytes.
__device__ __forceinline__ int blk_swz(int j) { return (j ^ (j >> 3)) & 7; }  // j = r & 15

constexpr int kFp8Lag = 3;

template <int DT, int NT, int MT, int WN, int WM, int SLOTS>
__global__ __launch_bounds__(64 * WN * WM, 2) void fp8_block_gemm(Fp8BlockArgs g, f32x4 *__restrict__ part) {
    constexpr int WAVES = WN * WM, BN = 16 * NT * WN, BM = 16 * MT * WM;
    constexpr int W_BYTES = BN * kBlk, A_BYTES = BM * kBlk, STAGE = W_BYTES + A_BYTES;
    constexpr int S_BYTES = BM * 16 + 64, LDS = SLOTS * STAGE + 2 * S_BYTES;
    constexpr int W_COPIES = BN / 8 / WAVES, A_COPIES = BM / 8 / WAVES, COPIES = W_COPIES + A_COPIES;
    static_assert(MT % 2 == 0 && kBlk % (16 * NT) == 0 && BM / 64 < WAVES && BN / kBlk <= 4 && LDS <= 163840, "fits");
    static_assert(SLOTS <= 4 && COPIES <= 2 * NT && (SLOTS - 1) * COPIES < 16, "two copies beside each weight operand at most; the wait's field");
    __shared__ __attribute__((aligned(16))) unsigned char lds[LDS];
    const int lane = threadIdx.x & 63, j = lane & 15, gq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const GroupMap map(g.groups, BM, (g.N + BN - 1) / BN);
    if ((int)blockIdx.x >= map.tiles()) return;
    const Fp8Tile t = fp8_tile(g, map.at(tile_of_xcd_order(blockIdx.x, map.tiles())), BM);
    const int K = g.K, N = g.N, blocks = (K + kBlk - 1) / kBlk;
    const int n0 = t.tile_n * BN;
    // this workgroup's stages; a K split begins at a multiple of four, where scales are copied
    const int S = gridDim.y, quarters = (blocks + 3) / 4;
    const int s_lo = 4 * (quarters * (int)blockIdx.y / S), s_hi = min(blocks, 4 * (quarters * ((int)blockIdx.y + 1) / S));
    const __amdgpu_buffer_rsrc_t wr = buf_rsrc(t.w + (size_t)n0 * K, (int64_t)min(BN, N - n0) * K);
    const __amdgpu_buffer_rsrc_t ar = buf_rsrc(t.a, (int64_t)t.a_rows * K);
    // waves 0 .. BM / 64 - 1 copy the tokens' scales, the next one the weights'
    const bool row_scales = wave < BM / 64, scales = wave <= BM / 64;
    const __amdgpu_buffer_rsrc_t sr = row_scales
        ? buf_rsrc(t.sa, (int64_t)t.a_rows * blocks * 4)
        : buf_rsrc(t.sw, (int64_t)((N + kBlk - 1) / kBlk) * blocks * 4);
    // Copies of 1 KB: 8 rows from row 8 c, lane % 8 being the stored segment of row 8 c + lane / 8.  Rows past
    // the matrices, and segments past K, are past the buffers: they read as zero.
    const int seg0 = (lane & 7) ^ (lane >> 3);
    uint32_t off[COPIES], so = kOut;
#pragma unroll
    for (int i = 0; i < W_COPIES; ++i) {
        const int c = wave * W_COPIES + i;
        off[i] = (uint32_t)((8 * c + (lane >> 3)) * K + 16 * (seg0 ^ (c & 1)));
    }
#pragma unroll
    for (int i = 0; i < A_COPIES; ++i) {
        const int c = wave * A_COPIES + i;
        const int src = fp8_source(g, t, 8 * c + (lane >> 3));
        off[W_COPIES + i] = src < 0 ? kOut : (uint32_t)src * (uint32_t)K + 16 * (seg0 ^ (c & 1));
    }
    if (row_scales) {
        const int src = fp8_source(g, t, 64 * wave + lane);
        if (src >= 0) so = (uint32_t)src * (uint32_t)blocks * 4u;
    } else if (wave == BM / 64 && lane < BN / kBlk) {
        so = (uint32_t)((n0 / kBlk + lane) * blocks) * 4u;
    }
    // copy i of stage st, whose rows have `left` 16-byte segments (none past the last stage; the wave's offset then
    // stays inside the buffers)
    auto copy1 = [&](int st, int slot, int left, auto ic) {
        constexpr int i = decltype(ic)::value;
        constexpr bool isw = i < W_COPIES;
        unsigned char *const dst = lds + slot * STAGE + (isw ? 0 : W_BYTES) +
                                   (wave * (isw ? W_COPIES : A_COPIES) + (isw ? i : i - W_COPIES)) * 1024;
        const int c = wave * (isw ? W_COPIES : A_COPIES) + (isw ? i : i - W_COPIES);
        dma16_buf(isw ? wr : ar, (seg0 ^ (c & 1)) < left ? off[i] : kOut, left ? (uint32_t)st * kBlk : 0u, dst);
    };
    auto copy_scales = [&](int st) {
        if (scales && (st & 3) == 0 && st < s_hi && (row_scales || lane < BN / kBlk))
            // (four scales may reach past the last row's: past the buffer)
            dma16_buf(sr, so + (uint32_t)st * 4u, 0u, lds + SLOTS * STAGE + ((st >> 2) & 1) * S_BYTES + (row_scales ? wave * 1024 : BM * 16));
    };
    auto left_of = [&](int st) { return st < s_hi ? min((K - st * kBlk) / 16, 8) : 0; };

    f32x4 acc[NT][MT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[i][m] = (f32x4){0.f, 0.f, 0.f, 0.f};
    const int a0 = j * kBlk + 16 * ((2 * gq) ^ blk_swz(j)), a1 = j * kBlk + 16 * ((2 * gq + 1) ^ blk_swz(j));
    auto operand = [&](int slot, int first, int tile) {
        const unsigned char *p = lds + slot * STAGE + first + tile * 16 * kBlk;
        return operand32(*(const u32x4 *)(p + a0), *(const u32x4 *)(p + a1));
    };
    auto row_scale = [&](int st, int m) {
        return *(const float *)(lds + SLOTS * STAGE + ((st >> 2) & 1) * S_BYTES + 16 * (16 * (wm * MT + m) + j) + 4 * (st & 3));
    };
    auto col_scale = [&](int st) {
        return *(const float *)(lds + SLOTS * STAGE + ((st >> 2) & 1) * S_BYTES + BM * 16 + 16 * (wn * NT * 16 / kBlk) + 4 * (st & 3));
    };
    {
        copy_scales(s_lo);
        static_for<SLOTS>([&](auto sc) {
            constexpr int slot = decltype(sc)::value;
            const int left = left_of(s_lo + slot);
            static_for<COPIES>([&](auto ic) { copy1(s_lo + slot, slot, left, ic); });
        });
        __builtin_amdgcn_s_waitcnt(0x0F70 | (SLOTS - 1) * COPIES);  // the first stage's have landed
        asm volatile("s_barrier" ::: "memory");
    }
    i32x8 w[NT], b[2];
    float sa[MT], sw;
#pragma unroll
    for (int i = 0; i < NT; ++i) w[i] = operand(0, 0, wn * NT + i);
    b[0] = operand(0, W_BYTES, wm * MT);
#pragma unroll
    for (int m = 0; m < MT; ++m) sa[m] = row_scale(s_lo, m);
    sw = col_scale(s_lo);
    int slot = 0;
    for (int st = s_lo; st < s_hi; ++st, slot = slot + 1 == SLOTS ? 0 : slot + 1) {
        const int left = left_of(st + SLOTS), next = slot + 1 == SLOTS ? 0 : slot + 1;
        constexpr int LAG = kFp8Lag, TILES = NT * MT;
        f32x4 p[LAG + 1];
        float sc[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) sc[m] = sa[m] * sw;
        static_for<TILES + LAG>([&](auto c) {
            constexpr int s = decltype(c)::value;
            if constexpr (s < TILES) {
                constexpr int m = s / NT, i = s % NT;
                if constexpr (m == MT - 1 && i == 0) {
                    // every operand of this stage is in registers and the next one's data have landed
                    __builtin_amdgcn_s_waitcnt(0x0070 | (SLOTS - 2) * COPIES);  // vmcnt, lgkmcnt(0)
                    asm volatile("s_barrier" ::: "memory");
                    copy_scales(st + SLOTS);
                }
                if constexpr (i == 0) {
                    if constexpr (m + 1 < MT) b[(m + 1) & 1] = operand(slot, W_BYTES, wm * MT + m + 1);
                    __builtin_amdgcn_sched_barrier(0);
                }
                p[s % (LAG + 1)] = mfma_fp8(w[i], b[m & 1], (f32x4){0.f, 0.f, 0.f, 0.f});
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (m == MT - 1) {
                    w[i] = operand(next, 0, wn * NT + i);
                    if constexpr (i == 0) {
                        b[0] = operand(next, W_BYTES, wm * MT);
                    }
                    static_assert(MT <= NT, "a token scale beside each");
                    if constexpr (i < MT) sa[i] = row_scale(st + 1, i);
                    if constexpr (i == NT - 1) sw = col_scale(st + 1);
                    if constexpr (i < COPIES) copy1(st + SLOTS, slot, left, std::integral_constant<int, i>{});
                    if constexpr (i + NT < COPIES) copy1(st + SLOTS, slot, left, std::integral_constant<int, i + NT>{});
                }
            }
            if constexpr (s >= LAG) {
                constexpr int m = (s - LAG) / NT, i = (s - LAG) % NT;
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][m][r] = __builtin_fmaf(p[(s - LAG) % (LAG + 1)][r], sc[m], acc[i][m][r]);
                asm volatile("" : "+v"(acc[i][m]));
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    }
    wait_vm_all();
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int row = 16 * (wm * MT + m) + j;
        if (row >= t.rows) continue;
        const size_t at = (size_t)(t.row0 + row) * N;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int n = n0 + 16 * (wn * NT + i) + 4 * gq;
            if (n >= N) continue;
            if (S == 1) *(uint2 *)((uint16_t *)g.y + at + n) = quad_out_bits<DT>(acc[i][m]);
            else part[((size_t)blockIdx.y * g.M * N + at + n) / 4] = acc[i][m];
        }
    }
}

template <int NT, int MT, int WN, int WM, int SLOTS>
static hipError_t launch_t(const Fp8BlockArgs &g, const Fp8BlockPlan &p, hipStream_t st) {
    const dim3 grid((unsigned)(p.tiles_n * p.tiles_m), (unsigned)p.splits), block(64 * WN * WM);
    f32x4 *const part = (f32x4 *)p.acc;
    if (g.dtype == DT_BF16) hipLaunchKernelGGL((fp8_block_gemm<DT_BF16, NT, MT, WN, WM, SLOTS>), grid, block, 0, st, g, part);
    else hipLaunchKernelGGL((fp8_block_gemm<DT_F16, NT, MT, WN, WM, SLOTS>), grid, block, 0, st, g, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    return launch_split_sum(part, g.y, g.groups.offsets, g.groups.E, g.M, g.N, p.splits, g.dtype, st);
}

hipError_t launch_fp8_block_gemm(const Fp8BlockArgs &g, const Fp8BlockPlan &p, hipStream_t st) {
    if (p.splits > 1 && p.acc == nullptr) return hipErrorInvalidValue;
    if (p.rows == 128 && p.cols == 128) return launch_t<4, 2, 2, 4, 4>(g, p, st);
    if (p.rows == 128 && p.cols == 256) return launch_t<4, 4, 4, 2, 3>(g, p, st);
    if (p.rows == 256 && p.cols == 256) return launch_t<8, 4, 2, 4, 2>(g, p, st);
    return hipErrorInvalidValue;
}

}  // namespace awq4
