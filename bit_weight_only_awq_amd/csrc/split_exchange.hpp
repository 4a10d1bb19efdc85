// split_exchange.hpp -- the end of the streaming kernels (stream_w4a16.hip,
// moe_w4a16.hip, stream_fp8_block.hip): the waves' tiles added, and the K splits' sums with
// them.
#pragma once

#include "device.hpp"
#include "launch.hpp"

namespace awq4 {

// Position of column c inside a parked row.  Lane j holds columns 8j .. 8j+7
// of its rows and parks them as two 16-byte halves: half h of every lane sits
// in the h-th half of the row, at the lane's 16-byte slot (4j floats), so the
// 16 lanes of a row write 16 consecutive slots -- all of the LDS banks, no
// two lanes of a write on one bank.  (Columns in plain order put lanes j and
// j+8 on the same banks and the four row groups of a wave on the same ones
// again: eight-way conflicts.)
template <int COLS>
__device__ __forceinline__ int lds_col(int c) {
    return (COLS / 2) * ((c >> 2) & 1) + 4 * (c >> 3) + (c & 3);
}

// The workgroup's M x COLS tile sum -- the SLOTS tiles its waves parked in
// LDS (ROWS rows of PITCH floats each, column c of a row at slot_of(c)), added
// in slot order -- goes out: written directly when the K range is not split
// (S == 1); otherwise handed over as fp32 partials (one M x N array per
// split after the tile counters), added in split order -- by the reduction
// kernel launched next where they are large (sep), else by the last
// workgroup of the column tile (device.hpp: split_tile_last_atomic), which
// also clears them and writes the output.  Everything moves as quads of columns (N is a
// multiple of 8, so a quad never straddles the last column): 8-byte output
// stores, 16-byte partial loads and stores.  The partials move with the
// cache policy of agent-scope atomic loads and stores (sc1: through to the
// device-wide coherence point), as 16-byte buffer accesses -- half the
// requests of 8-byte atomics; the tail of the kernel is the last workgroups'
// partial traffic, so its request count sets the tail's length.

// M: rows of the tile that exist.  Where it begins at a row of a larger output
// (products grouped by expert), y and part point at that row, slot_bytes is
// from one split's partials to the next, and cnt is the tile's own counter.
template <int NT, int DT, int ROWS, int COLS, int PITCH, int SLOTS, class SlotOf>
__device__ __forceinline__ void tile_store_or_exchange(const float *red, SlotOf slot_of, uint16_t *__restrict__ y,
                                                       uint32_t *cnt, char *part, size_t slot_bytes, int M, int N,
                                                       int tile, int S, int sep) {
    constexpr int QR = COLS / 4;         // quads per row
    constexpr int kQ = (ROWS * QR + NT - 1) / NT;  // quads per thread, whole tile
    const int n_base = tile * COLS;
    const int quads = M * QR;
    // thread t takes quads t, t + NT, ...: its sums of the SLOTS parked tiles
    // and their 16-byte index in an [M, N] array
    f32x4 v[kQ];
    bool ok[kQ];
    uint32_t at[kQ];
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
        const int qi = threadIdx.x + q * NT;
        const int r = qi / QR, c = 4 * (qi % QR);
        ok[q] = qi < quads && n_base + c < N;
        at[q] = ok[q] ? (uint32_t)(r * (N / 4) + (n_base + c) / 4) : 0u;
        v[q] = (f32x4){0.f, 0.f, 0.f, 0.f};
        if (ok[q]) {
            const float *p = red + r * PITCH + slot_of(c);
            v[q] = *(const f32x4 *)p;
#pragma unroll
            for (int w = 1; w < SLOTS; ++w) v[q] += *(const f32x4 *)(p + w * ROWS * PITCH);
        }
    }
    auto out_quad = [&](uint32_t a, f32x4 t) { *(uint2 *)(y + 4 * (size_t)a) = quad_out_bits<DT>(t); };
    if (S == 1) {
#pragma unroll
        for (int q = 0; q < kQ; ++q)
            if (ok[q]) out_quad(at[q], v[q]);
        return;
    }
    // split s's partials: a buffer over its M x N floats (under 2^31 bytes,
    // which the planner ensures)
    const uint32_t tile_bytes = (uint32_t)M * (uint32_t)N * 4u;
    auto split_rsrc = [&](int s) { return buf_rsrc(part + (size_t)s * slot_bytes, tile_bytes); };
    const int own = blockIdx.y;
    // sep: the reduction kernel launched next adds the splits (plain stores,
    // made visible by the kernel boundary); else the column tile's last
    // workgroup adds them below.
    {
        const __amdgpu_buffer_rsrc_t rs = split_rsrc(own);
#pragma unroll
        for (int q = 0; q < kQ; ++q)
            if (ok[q]) {
                if (sep) __builtin_amdgcn_raw_buffer_store_b128(bit_as<u32x4>(v[q]), rs, at[q] * 16u, 0, 0);
                else __builtin_amdgcn_raw_buffer_store_b128(bit_as<u32x4>(v[q]), rs, at[q] * 16u, 0, kPartCoherent);
            }
    }
    if (sep || !split_tile_last_atomic(cnt, S)) return;
    // The last workgroup of the column tile: the other splits' partials of
    // all its quads, kB splits at a time with every load of a batch issued
    // before the first add (one memory round trip per batch), added in split
    // order with its own partial (still in registers) in its place.
    constexpr int kB = 32 / kQ < 1 ? 1 : 32 / kQ > 8 ? 8 : 32 / kQ;
    f32x4 sum[kQ];
#pragma unroll
    for (int q = 0; q < kQ; ++q) sum[q] = (f32x4){0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < S; s0 += kB) {
        u32x4 b[kQ][kB];
#pragma unroll
        for (int i = 0; i < kB; ++i) {
            const int s = s0 + i;
#pragma unroll
            for (int q = 0; q < kQ; ++q) b[q][i] = (u32x4){0u, 0u, 0u, 0u};
            if (s < S && s != own) {
                const __amdgpu_buffer_rsrc_t rs = split_rsrc(s);
#pragma unroll
                for (int q = 0; q < kQ; ++q)
                    if (ok[q]) b[q][i] = __builtin_amdgcn_raw_buffer_load_b128(rs, at[q] * 16u, 0, kPartCoherent);
            }
        }
#pragma unroll
        for (int i = 0; i < kB; ++i) {
            const int s = s0 + i;
            if (s >= S) break;
#pragma unroll
            for (int q = 0; q < kQ; ++q) sum[q] += s == own ? v[q] : bit_as<f32x4>(b[q][i]);
        }
    }
    for (int s = 0; s < S; ++s) {
        const __amdgpu_buffer_rsrc_t rs = split_rsrc(s);
#pragma unroll
        for (int q = 0; q < kQ; ++q)
            if (ok[q]) __builtin_amdgcn_raw_buffer_store_b128((u32x4){0u, 0u, 0u, 0u}, rs, at[q] * 16u, 0, kPartCoherent);
    }
#pragma unroll
    for (int q = 0; q < kQ; ++q)
        if (ok[q]) out_quad(at[q], sum[q]);
}

}  // namespace awq4
