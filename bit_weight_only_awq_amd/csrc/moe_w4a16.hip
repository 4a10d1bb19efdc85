// moe_w4a16.hip -- AWQ W4A16 products grouped by expert, for few rows an expert:
// every expert's weights are streamed once, straight into registers.
//
// Method as in w4a16.hip.  A workgroup has 256 outputs of one expert and a tile
// of 16 MT of its rows; its four waves take the chunks of 32 CS consecutive k (inside
// one quantisation group) in turn -- with a K split, of the workgroup's share of
// them -- with two chunks' loads in flight, and their sums are added through LDS in wave
// order, then over the K splits in split order (split_exchange.hpp).  (The four tiles of
// 32 rows are 128 KB of LDS: one workgroup a CU, where 16 rows leave room for two.)
//
// Lane (j, gq) holds two neighbouring word-columns (16 outputs) at the 8 k-rows 8 gq + e
// of each 32-k step: a load takes whole 128-byte lines of four k-rows.  That sets the
// rate: two experts' 4096 x 28672 (117 MB) read alone in 22 us so, 30 to 35 us by lanes of one
// word-column, whose lines two workgroups share, and the same in any order of them.
// (Shares of equal length for every workgroup over all tiles' chunks, wherever a tile ends,
// brought no more than that order lost: 18 us for the smallest call against 5.)
//
// The weights enter the matrix cores without arithmetic: a pair of nibbles masked
// out of two paired words is a pair of fp16 subnormals q 2^-24 (16 q 2^-24 for an
// upper nibble), or ORed into the mantissa of 128.0 the pair of bf16 numbers 128 + q;
// both exact.  Scale and zero point are applied to a chunk's fp32 sums, s (sum x q - z
// sum x), with sum x from one more matrix-core instruction against ones.  That is
// one bitwise operation a pair, against two (fp16) and six (bf16) for the exact q - z:
// what a stream at the memory's rate leaves time for.  Where an infinity in x meets q = 0, or both sums pass
// binary32 on the way to a difference that does not, a wave's sums come out infinite or NaN: it then makes them again from the
// exact q - z, whose sums are those of the definition (a token with an infinity, 4096 x 28672 of two experts: 41 us, not 32).
#include "moe.hpp"
#include "split_exchange.hpp"
#include "w4a16_ops.hpp"

namespace awq4 {

template <int MT, int CS>
struct GroupedBuf {
    u32x4 s4[2];
    u32x2 zw;
    u32x4 a[MT][CS];
    u32x2 w[CS][8];
};

// One word-column of the chunk into its eight outputs' sums; NR: 4, or 1 where the tile has one row (a lane's rows are
// 4 gq + r, so the first r of 0 .. 3 are all that a tile of r rows needs).
template <int MT, int CS, int DT, bool SYM, int NR>
__device__ __forceinline__ void grouped_column(const GroupedBuf<MT, CS> &b, int col, const f32x4 (&rs)[MT],
                                               f32x4 (&acc)[MT][8]) {
    uint32_t px[CS][4], py[CS][4];
#pragma unroll
    for (int s = 0; s < CS; ++s)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            px[s][p] = pair_x(b.w[s][2 * p][col], b.w[s][2 * p + 1][col]);
            py[s][p] = pair_y(b.w[s][2 * p][col], b.w[s][2 * p + 1][col]);
        }
    static_for<8>([&](auto tc) {
        constexpr int T = decltype(tc)::value;
        f32x4 t[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) t[m] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < CS; ++s) {
            u32x4 bop;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint32_t v = col_src_y(T) ? py[s][p] : px[s][p];
                if constexpr (DT == DT_F16)
                    bop[p] = (col_shift(T) ? v >> 8 : v) & (col_hi(T) ? 0x00F000F0u : 0x000F000Fu);
                else
                    bop[p] = __builtin_amdgcn_bitop3_b32(v >> (col_shift(T) + 4 * col_hi(T)), 0x000F000Fu, 0x43004300u, 0xEA);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) t[m] = mma<DT>(b.a[m][s], bop, t[m]);
        }
        const float st = scale_f32<DT>(b.s4[col], T);
        const float zt = SYM ? 8.0f : (float)((b.zw[col] >> (4 * col_nibble(T))) & 0xFu);
        const float at = DT == DT_F16 ? st * (col_hi(T) ? 0x1p20f : 0x1p24f) : st;
        const float bt = -st * (DT == DT_F16 ? zt : 128.0f + zt);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < NR; ++r)
                acc[m][T][r] = __builtin_fmaf(t[m][r], at, __builtin_fmaf(bt, rs[m][r], acc[m][T][r]));
        // four columns at a time: bounds how many temporaries are live at once
        if (T % 4 == 3) __builtin_amdgcn_sched_barrier(0);
    });
}

// The same by the exact q - z.
template <int MT, int CS, int DT, bool SYM>
__device__ __forceinline__ void grouped_column_exact(const GroupedBuf<MT, CS> &b, int col, f32x4 (&acc)[MT][8]) {
    ZeroConsts<DT> zc;
    zero_consts<DT, SYM>(zc, SYM ? 0u : b.zw[col]);
    static_for<8>([&](auto tc) {
        constexpr int T = decltype(tc)::value;
        f32x4 t[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) t[m] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < CS; ++s) {
            u32x4 bop;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint32_t w0 = b.w[s][2 * p][col], w1 = b.w[s][2 * p + 1][col];
                bop[p] = qz_pair<DT, T>(col_src_y(T) ? pair_y(w0, w1) : pair_x(w0, w1), zc);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) t[m] = mma<DT>(b.a[m][s], bop, t[m]);
        }
        const float st = scale_f32<DT>(b.s4[col], T);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[m][T][r] = __builtin_fmaf(t[m][r], st, acc[m][T][r]);
        __builtin_amdgcn_sched_barrier(0);
    });
}

template <int MT, int CS, int DT, bool SYM>
__global__ __launch_bounds__(64 * kGroupedWaves, 2) void w4a16_grouped(
    const uint16_t *__restrict__ x, const uint32_t *__restrict__ qw, const uint16_t *__restrict__ sc,
    const uint32_t *__restrict__ qz, uint16_t *__restrict__ y, uint64_t *__restrict__ ws, int N, int K, int lgG,
    Groups grp) {
    constexpr int WV = kGroupedWaves, ROWS = 16 * MT, COLS = kGroupedCols;
    __shared__ __attribute__((aligned(16))) float red[WV * ROWS * COLS];
    const int lane = threadIdx.x & 63, j = lane & 15, gq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nw = N >> 3, groups = K >> lgG;
    const GroupMap map(grp, ROWS, (N + COLS - 1) / COLS);
    if ((int)blockIdx.x >= map.tiles()) return;
    const int index = tile_of_xcd_order(blockIdx.x, map.tiles());
    const GroupTile t = map.at(index);
    const int rows = min(t.row_end - t.row0, ROWS);
    const size_t e = t.expert;
    // this workgroup's chunks [lo, hi) and this wave's share of them
    const int S = gridDim.y, chunks = K / (32 * CS), per = (chunks + S - 1) / S;
    const int lo = blockIdx.y * per, hi = min(chunks, lo + per);
    const int n = hi - lo > wave ? (hi - lo - wave + WV - 1) / WV : 0;
    // (an expert's weights, and gathered rows, are under 2^31 bytes.)  Columns past the last are past the buffers:
    // nothing is loaded for them, and rows past the tile's read its first: neither's sums are stored.  (Nor are those of
    // the second word-column of a row's last pair where N / 8 is odd: the next row's first, or past the buffer.)
    const __amdgpu_buffer_rsrc_t qr = buf_rsrc(qw + e * K * nw, (int64_t)K * nw * 4);
    const __amdgpu_buffer_rsrc_t sr = buf_rsrc(sc + e * groups * N, (int64_t)groups * N * 2);
    const __amdgpu_buffer_rsrc_t zr = buf_rsrc(SYM ? qw : qz + e * groups * nw, SYM ? 0 : (int64_t)groups * nw * 4);
    const __amdgpu_buffer_rsrc_t xr = buf_rsrc(grp.rows ? x : x + (size_t)t.row0 * K,
                                               (int64_t)(grp.rows ? grp.x_rows : rows) * K * 2);
    const int wcol = t.tile_n * (COLS / 8) + 2 * j;
    const bool have = wcol < nw;
    const uint32_t ow = have ? (uint32_t)(8 * gq * nw + wcol) * 4u : 0x80000000u;
    const uint32_t os = have ? (uint32_t)wcol * 16u : 0x80000000u, oz = have ? (uint32_t)wcol * 4u : 0x80000000u;
    uint32_t ox[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        int src = 16 * m + j < rows ? 16 * m + j : 0;
        if (grp.rows) src = group_source(grp.rows, t.row0 + src, grp.top, grp.x_rows);
        ox[m] = (uint32_t)src * (uint32_t)K * 2u + 16u * gq;
    }
    auto issue = [&](GroupedBuf<MT, CS> &b, int i) {
        const uint32_t k0 = (lo + wave + i * WV) * 32 * CS, g = k0 >> lgG;
        uint32_t at = k0 * nw * 4;
#pragma unroll
        for (int s = 0; s < CS; ++s) {
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                b.w[s][r] = __builtin_amdgcn_raw_buffer_load_b64(qr, ow, at, 2);  // (read once: non-temporal)
                at += nw * 4;
            }
            at += 24 * nw * 4;
        }
        b.s4[0] = __builtin_amdgcn_raw_buffer_load_b128(sr, os, g * N * 2, 0);
        b.s4[1] = __builtin_amdgcn_raw_buffer_load_b128(sr, os + 16, g * N * 2, 0);
        if (!SYM) b.zw = __builtin_amdgcn_raw_buffer_load_b64(zr, oz, g * nw * 4, 0);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int s = 0; s < CS; ++s) b.a[m][s] = __builtin_amdgcn_raw_buffer_load_b128(xr, ox[m] + 64 * s, k0 * 2, 0);
        // keeps the loads where they are issued, two chunks ahead of their use
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    f32x4 acc[2][MT][8];
    auto clear = [&] {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int u = 0; u < 8; ++u) acc[c][m][u] = (f32x4){0.f, 0.f, 0.f, 0.f};
    };
    clear();
    auto run = [&](auto nr) {
        auto compute = [&](const GroupedBuf<MT, CS> &b) {
            constexpr uint32_t one = DT == DT_F16 ? 0x3C003C00u : 0x3F803F80u;
            f32x4 rs[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                rs[m] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < CS; ++s) rs[m] = mma<DT>(b.a[m][s], (u32x4){one, one, one, one}, rs[m]);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) grouped_column<MT, CS, DT, SYM, decltype(nr)::value>(b, c, rs, acc[c]);
        };
        GroupedBuf<MT, CS> b0, b1;
        if (n > 0) issue(b0, 0);
        if (n > 1) issue(b1, 1);
        int i = 0;
        for (; i + 3 < n; i += 2) {
            compute(b0);
            issue(b0, i + 2);
            compute(b1);
            issue(b1, i + 3);
        }
        if (i < n) compute(b0);
        if (i + 2 < n) issue(b0, i + 2);
        if (i + 1 < n) compute(b1);
        if (i + 2 < n) compute(b0);
        // 0 while every sum is finite (an infinity or a NaN stays in its sum)
        f32x4 odd = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int u = 0; u < 8; ++u)
#pragma unroll
                    for (int r = 0; r < decltype(nr)::value; ++r) odd[u & 3] = __builtin_fmaf(acc[c][m][u][r], 0.0f, odd[u & 3]);
        if (__ballot((odd[0] + odd[1]) + (odd[2] + odd[3]) != 0.0f) == 0) return;
        clear();
#pragma unroll 1
        for (i = 0; i < n; ++i) {
            issue(b0, i);
#pragma unroll
            for (int c = 0; c < 2; ++c) grouped_column_exact<MT, CS, DT, SYM>(b0, c, acc[c]);
        }
    };
    if (MT == 1 && rows == 1) run(std::integral_constant<int, 1>{});
    else run(std::integral_constant<int, 4>{});

    // lane: rows 16 m + 4 gq + r, columns 16 j + 8 c + u of the tile; quad q of a lane's 16 columns at 64 q + 4 j, so
    // that the 16 lanes of a row write consecutive slots
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float *d = red + ((size_t)wave * ROWS + 16 * m + 4 * gq + r) * COLS + 4 * j;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4(&v)[8] = acc[q >> 1][m];
                const int u = 4 * (q & 1);
                *(f32x4 *)(d + 64 * q) = (f32x4){v[u][r], v[u + 1][r], v[u + 2][r], v[u + 3][r]};
            }
        }
    __syncthreads();
    const size_t at = (size_t)t.row0 * N;
    tile_store_or_exchange<64 * WV, DT, ROWS, COLS, COLS, WV>(
        red, [](int c) { return 64 * ((c >> 2) & 3) + 4 * (c >> 4) + (c & 3); }, y + at, (uint32_t *)ws + index,
        (char *)ws + split_counters_bytes(gridDim.x) + at * 4, (size_t)grp.R * N * 4, rows, N, t.tile_n, S, 0);
}

template <int MT, int CS, int DT, bool SYM>
static hipError_t launch_t(const W4A16Args &a, const W4A16Plan &p, const Groups &g, hipStream_t st) {
    hipLaunchKernelGGL((w4a16_grouped<MT, CS, DT, SYM>), dim3((unsigned)(p.tiles_n * p.tiles_m), p.splits),
                       dim3(64 * kGroupedWaves), 0, st, (const uint16_t *)a.x, (const uint32_t *)a.qweight,
                       (const uint16_t *)a.scales, (const uint32_t *)a.qzeros, (uint16_t *)a.y, p.acc, (int)a.N,
                       (int)a.K, __builtin_ctz((unsigned)a.G), g);
    return hipGetLastError();
}

template <int MT, int CS>
static hipError_t launch_dt(const W4A16Args &a, const W4A16Plan &p, const Groups &g, hipStream_t st) {
    const bool sym = a.qzeros == nullptr;
    if (a.dtype == DT_F16)
        return sym ? launch_t<MT, CS, DT_F16, true>(a, p, g, st) : launch_t<MT, CS, DT_F16, false>(a, p, g, st);
    return sym ? launch_t<MT, CS, DT_BF16, true>(a, p, g, st) : launch_t<MT, CS, DT_BF16, false>(a, p, g, st);
}

// p.mt: 16-row tiles (1, 2); p.cs: 32-k steps of a chunk (1, 2)
hipError_t launch_w4a16_grouped(const W4A16Args &a, const W4A16Plan &p, const Groups &g, hipStream_t st) {
    if ((p.splits > 1 && p.acc == nullptr) || 32 * p.cs > a.G) return hipErrorInvalidValue;
    switch (p.mt * 10 + p.cs) {
        case 11: return launch_dt<1, 1>(a, p, g, st);
        case 12: return launch_dt<1, 2>(a, p, g, st);
        case 21: return launch_dt<2, 1>(a, p, g, st);
        case 22: return launch_dt<2, 2>(a, p, g, st);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace awq4
