// gemm_fp8_block.hip -- block-scaled E4M3 products of many rows (fp8_block.hpp
// has the arithmetic): tiles through LDS.
//
// A workgroup of 8 waves has BN outputs n and BM tokens, a wave NT x MT tiles of
// 16 x 16 of them.  A stage is one block of 128 k: the rows of both matrices (128
// bytes of each) and the block's scales are copied straight into LDS, one
// stage ahead.  The matrix cores' sum of a tile and block is scaled and added
// to the running sums two matrix-core instructions later, so that a wave
// issues the next ones while it waits for none: four FMAs beside every
// instruction of 32 cycles.
#include "fp8_block.hpp"

namespace awq4 {

// 4 bytes a lane, as dma16_buf
__device__ __forceinline__ void dma4_buf(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, void *dst) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 :
                 : "s"(lds_address(dst)), "v"(voff), "s"(r), "s"(soff)
                 : "memory", "m0");
}

// 16-byte segment s of row r is stored at s ^ blk_swz(r): the 16 rows of an
// operand read lie on 16 different bank groups of 256 bytes.
__device__ __forceinline__ int blk_swz(int r) { return (r ^ (r >> 3)) & 7; }

template <int BM, int BN, int WM, int RING>
struct Fp8Lds {
    static constexpr int WN = 8 / WM;
    static constexpr int NT = BN / WN / 16, MT = BM / WM / 16;
    static constexpr int W_BYTES = BN * kBlk, A_BYTES = BM * kBlk;
    static constexpr int S_BYTES = BM * 4 + 16;  // token scales, then the weights' (up to 4)
    static constexpr int STAGE = W_BYTES + A_BYTES + S_BYTES;
    static constexpr int LDS = RING * STAGE;
    static constexpr int W_COPIES = BN / 64, A_COPIES = BM / 64;  // 1 KB copies of a wave and stage
    static_assert(LDS <= 163840 && BN % 128 == 0 && BM % 64 == 0 && (BN / WN) % 16 == 0, "fits");
};

template <int DT, int BM, int BN, int WM, int RING>
__global__ __launch_bounds__(512, 2) void fp8_block_gemm(Fp8BlockArgs g) {
    using L = Fp8Lds<BM, BN, WM, RING>;
    constexpr int NT = L::NT, MT = L::MT;
    __shared__ __attribute__((aligned(16))) unsigned char lds[L::LDS];
    const int lane = threadIdx.x & 63, j = lane & 15, gq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const Fp8Tile t = fp8_tile(g, BM, BN, blockIdx.x);
    if (!t.live) return;
    const int K = g.K, N = g.N, blocks = (K + kBlk - 1) / kBlk;
    const int n0 = t.tile_n * BN;

    // rows past the matrices, and k past K, are past the buffers: they read as zero
    const __amdgpu_buffer_rsrc_t wr = buf_rsrc(t.w + (size_t)n0 * K, (int64_t)min(BN, N - n0) * K);
    const __amdgpu_buffer_rsrc_t ar = buf_rsrc(t.a, (int64_t)t.a_rows * K);
    const __amdgpu_buffer_rsrc_t sr = buf_rsrc(t.sa, (int64_t)t.a_rows * blocks * 4);
    const __amdgpu_buffer_rsrc_t vr =
        buf_rsrc(t.sw, (int64_t)((N + kBlk - 1) / kBlk) * blocks * 4);
    // Copies: copy i of wave w takes rows 8 (w C + i) + lane / 8, lane % 8 being the stored segment.
    const int seg0 = (lane & 7) ^ (lane >> 3);
    uint32_t wo[L::W_COPIES], ao[L::A_COPIES], so = kOut;
#pragma unroll
    for (int i = 0; i < L::W_COPIES; ++i) {
        const int c = wave * L::W_COPIES + i;
        wo[i] = (uint32_t)((8 * c + (lane >> 3)) * K + 16 * (seg0 ^ (c & 7)));
    }
#pragma unroll
    for (int i = 0; i < L::A_COPIES; ++i) {
        const int c = wave * L::A_COPIES + i;
        const int src = fp8_source(g, t, 8 * c + (lane >> 3));
        ao[i] = src < 0 ? kOut : (uint32_t)src * (uint32_t)K + 16 * (seg0 ^ (c & 7));
    }
    const bool scale_wave = wave < BM / 64, weight_wave = wave == 7;
    static_assert(BM / 64 <= 7, "wave 7 copies the weights' scales");
    if (scale_wave) {
        const int src = fp8_source(g, t, 64 * wave + lane);
        if (src >= 0) so = (uint32_t)src * (uint32_t)blocks * 4u;
    } else if (weight_wave && lane < BN / kBlk) {
        so = (uint32_t)((n0 / kBlk + lane) * blocks) * 4u;
    }
    auto copy = [&](int st, int slot) {
        unsigned char *const base = lds + slot * L::STAGE;
        const uint32_t k = (uint32_t)st * kBlk;
        unsigned char *const w = base + wave * L::W_COPIES * 1024, *const a = base + L::W_BYTES + wave * L::A_COPIES * 1024;
        const int left = (K - st * kBlk) / 16;  // 16-byte segments of a row that are left
        if (left >= 8) {
#pragma unroll
            for (int i = 0; i < L::W_COPIES; ++i) dma16_buf(wr, wo[i], k, w + i * 1024);
#pragma unroll
            for (int i = 0; i < L::A_COPIES; ++i) dma16_buf(ar, ao[i], k, a + i * 1024);
        } else {
#pragma unroll
            for (int i = 0; i < L::W_COPIES; ++i)
                dma16_buf(wr, (seg0 ^ ((wave * L::W_COPIES + i) & 7)) < left ? wo[i] : kOut, k, w + i * 1024);
#pragma unroll
            for (int i = 0; i < L::A_COPIES; ++i)
                dma16_buf(ar, (seg0 ^ ((wave * L::A_COPIES + i) & 7)) < left ? ao[i] : kOut, k, a + i * 1024);
        }
        unsigned char *const s = base + L::W_BYTES + L::A_BYTES;
        if (scale_wave) dma4_buf(sr, so, (uint32_t)st * 4u, s + wave * 256);
        else if (weight_wave && lane < BN / kBlk) dma4_buf(vr, so, (uint32_t)st * 4u, s + BM * 4);
    };

    f32x4 acc[NT][MT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[i][m] = (f32x4){0.f, 0.f, 0.f, 0.f};

    // operand of 16 rows from row r0: segments 2 gq and 2 gq + 1 of row r0 + j
    auto operand = [&](const unsigned char *base, int r0) {
        const int r = r0 + j;
        const unsigned char *p = base + r * kBlk;
        return operand32(*(const u32x4 *)(p + 16 * ((2 * gq) ^ blk_swz(r))),
                         *(const u32x4 *)(p + 16 * ((2 * gq + 1) ^ blk_swz(r))));
    };
    auto stage = [&](int st, int slot) {
        if (st + 1 < blocks) copy(st + 1, slot ^ 1);
        const unsigned char *const W = lds + slot * L::STAGE, *const A = W + L::W_BYTES, *const S = A + L::A_BYTES;
        i32x8 b[MT], w[3];
        float sc[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) b[m] = operand(A, 16 * (wm * MT + m));
        w[0] = operand(W, 16 * (wn * NT));
        w[1] = operand(W, 16 * (wn * NT + 1));
        const float sw = *(const float *)(S + BM * 4 + 4 * (wn * NT * 16 / kBlk));
#pragma unroll
        for (int m = 0; m < MT; ++m) sc[m] = *(const float *)(S + 4 * (16 * (wm * MT + m) + j)) * sw;
        constexpr int LAG = 2, TILES = NT * MT;
        f32x4 p[4];
        static_for<TILES + LAG>([&](auto c) {
            constexpr int s = decltype(c)::value;
            if constexpr (s < TILES) {
                constexpr int i = s / MT, m = s % MT;
                if constexpr (m == 0 && i + 2 < NT) w[(i + 2) % 3] = operand(W, 16 * (wn * NT + i + 2));
                p[s & 3] = mfma_fp8(w[i % 3], b[m], (f32x4){0.f, 0.f, 0.f, 0.f});
            }
            if constexpr (s >= LAG) {
                constexpr int i = (s - LAG) / MT, m = (s - LAG) % MT;
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][m][r] = __builtin_fmaf(p[(s - LAG) & 3][r], sc[m], acc[i][m][r]);
            }
            __builtin_amdgcn_sched_barrier(0);
        });
        wait_vm_all();
        asm volatile("s_barrier" ::: "memory");
    };
    static_assert((NT * 16) % kBlk == 0 || kBlk % (NT * 16) == 0, "a wave's columns lie in one block");
    copy(0, 0);
    wait_vm_all();
    __syncthreads();
    for (int st = 0; st < blocks; ++st) stage(st, st & 1);

    // lane: outputs n + r of token 16 m + j
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int row = 16 * (wm * MT + m) + j;
        if (row >= t.rows) continue;
        uint16_t *const y = (uint16_t *)g.y + (size_t)(t.row0 + row) * N;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int n = n0 + 16 * (wn * NT + i) + 4 * gq;
            if (n < N) *(uint2 *)(y + n) = quad_out_bits<DT>(acc[i][m]);
        }
    }
}

template <int BM, int BN, int WM, int RING>
static hipError_t launch_t(const Fp8BlockArgs &g, const Fp8BlockPlan &p, hipStream_t st) {
    const dim3 grid((unsigned)(p.tiles_n * p.tiles_m));
    if (g.dtype == DT_BF16)
        hipLaunchKernelGGL((fp8_block_gemm<DT_BF16, BM, BN, WM, RING>), grid, dim3(512), 0, st, g);
    else
        hipLaunchKernelGGL((fp8_block_gemm<DT_F16, BM, BN, WM, RING>), grid, dim3(512), 0, st, g);
    return hipGetLastError();
}

hipError_t launch_fp8_block_gemm(const Fp8BlockArgs &g, const Fp8BlockPlan &p, hipStream_t st) {
    if (p.splits != 1) return hipErrorInvalidValue;
    return launch_t<256, 256, 4, 2>(g, p, st);
}

}  // namespace awq4
