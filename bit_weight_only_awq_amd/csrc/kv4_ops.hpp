// kv4_ops.hpp -- what the kernels for few query rows (kv4_attention.hip,
// kv4_decode.hip) share: operands from packed words, exchanges within a column
// of scores, and the joining of partial sums.  Their mathematics is described
// in kv4_attention.hip.
#pragma once

#include "kv4.hpp"
#include "launch.hpp"

namespace awq4 {

constexpr int kAttnWaves = 4;
constexpr float kNoRef = -0x1.fffffep127f;  // the reference of a row that has seen nothing
constexpr float kMaxP = 0x1p15f, kMaxSum = 0x1p100f;
// From here on a reference is too coarse for the numerators to stay within
// fp16's range around it: such a row is NaN (a row of zeros would look like an answer).
constexpr float kFarRef = 0x1p25f;

// The reference of a row whose scores ask for m (-infinity: nothing seen).
// Scores of 2^24 and more come in steps of two and more, and m's roundings may
// leave it as far below what the numerators then are; from there on it is
// taken higher by as much, so that they never pass fp16's range.
__device__ __forceinline__ float raised(float ref, float m) {
    return fmaxf(ref, m + fmaxf(__builtin_fmaf(fabsf(m), 0x1p-22f, -4.0f), 0.0f));
}

// The larger of the values of the four lanes of a column (lanes l, l ^ 16, l ^
// 32, l ^ 48), in each of them.
__device__ __forceinline__ float column_max(float v) {
    const uint32_t b = bit_as<uint32_t>(v);
    const auto h = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const float m = fmaxf(bit_as<float>((uint32_t)h[0]), bit_as<float>((uint32_t)h[1]));
    const uint32_t c = bit_as<uint32_t>(m);
    const auto q = __builtin_amdgcn_permlane16_swap(c, c, false, false);
    return fmaxf(bit_as<float>((uint32_t)q[0]), bit_as<float>((uint32_t)q[1]));
}
__device__ __forceinline__ float column_sum(float v) {
    const uint32_t b = bit_as<uint32_t>(v);
    const auto h = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const float m = bit_as<float>((uint32_t)h[0]) + bit_as<float>((uint32_t)h[1]);
    const uint32_t c = bit_as<uint32_t>(m);
    const auto q = __builtin_amdgcn_permlane16_swap(c, c, false, false);
    return bit_as<float>((uint32_t)q[0]) + bit_as<float>((uint32_t)q[1]);
}

// The eight codes of a word as matrix-core operand (fp16 subnormals), columns
// 0..7 in order; columns 2, 3, 6, 7 carry a factor 16.
__device__ __forceinline__ u32x4 word_operand(uint32_t w) {
    return (u32x4){w & 0x000F000Fu, w & 0x00F000F0u, (w >> 8) & 0x000F000Fu, (w >> 8) & 0x00F000F0u};
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    return bit_as<uint32_t>(__builtin_convertvector((f32x2){a, b}, f16x2));
}

// Matrix-core operands from the value words of four tokens pairs (w[i]: pair
// i's words, consecutive tokens): operand t's rows are output dimensions
// value_dim(t, row).  A lane holds word column lane % 16 (D = 128: all eight
// columns of a word, one an operand) or lane % 8 (D = 64: the even columns in
// lanes 0..7 of a row of lanes, the odd ones in lanes 8..15).
template <int D>
__host__ __device__ constexpr int value_dim(int t, int row) {
    return D == 128 ? 8 * row + t : 8 * (row & 7) + 2 * t + (row >> 3);
}
template <int D>
__host__ __device__ constexpr int value_pos(int t) {  // nibble position in a 16-bit half
    return D == 128 ? t >> 1 : t;
}
// an operand counts in 2^-24, or 2^-20 where its nibbles are the upper ones of a byte
template <int D>
__host__ __device__ constexpr float value_unit(int t) {
    return value_pos<D>(t) & 1 ? 0x1p20f : 0x1p24f;
}
template <int D>
struct ValuePairs {
    uint32_t px[4], py[4];
    __device__ __forceinline__ ValuePairs(u32x4 first, u32x4 second, int r16) {
        const uint32_t half_sel = (D == 128 || r16 < 8) ? 0x05040100u : 0x07060302u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const u32x4 &w = i < 2 ? first : second;
            px[i] = perm_b32(w[2 * (i & 1) + 1], w[2 * (i & 1)], half_sel);
            py[i] = D == 128 ? pair_y(w[2 * (i & 1)], w[2 * (i & 1) + 1]) : 0u;
        }
    }
    __device__ __forceinline__ u32x4 operand(int t) const {
        const int pos = value_pos<D>(t);
        u32x4 a;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = D == 128 && (t & 1) ? py[i] : px[i];
            a[i] = (pos & 2 ? w >> 8 : w) & (pos & 1 ? 0x00F000F0u : 0x000F000Fu);
        }
        return a;
    }
};

// A lane's eight query values (fp32) as operand against word_operand: columns
// 2, 3, 6, 7 meet codes times 16.
__device__ __forceinline__ u32x4 query_operand(const float (&f)[8]) {
    return (u32x4){pack_f16(f[0], f[1]), pack_f16(f[2] * 0.0625f, f[3] * 0.0625f), pack_f16(f[4], f[5]),
                   pack_f16(f[6] * 0.0625f, f[7] * 0.0625f)};
}
// The power of two that takes a row whose largest magnitude is mx to just below 2^15.
__device__ __forceinline__ int query_shift(float mx) {
    const int ex = (int)(bit_as<uint32_t>(mx) >> 23);
    return ex == 255 || ex == 0 ? 0 : min(127 + 14 - ex, 100);
}

// What a tile of query rows (TILE of a sequence and key/value head, tile ct of
// them) reads, and how many workgroups share it; whatever the index arrays
// hold, no index made from it leaves the tensors.  All of it uniform.
template <int TILE, int STEP>
struct Kv4Span {
    int q0, nq, kv_len, c0, ncols;  // first row of the sequence, new tokens, length; the tile's rows (ncols <= 0: none)
    int kv_lo, kv_hi;               // tokens that any row of the tile sees
    int s_begin, steps, chunk, splits;  // first step of STEP tokens, number of steps, of them for a workgroup, of workgroups
    __device__ __forceinline__ Kv4Span(const Kv4AttnArgs &g, int b, int ct, int G) {
        q0 = b;
        int q1 = b + 1;
        if (g.cu_q) {
            q0 = min(max(g.cu_q[b], 0), g.total_q);
            q1 = min(max(g.cu_q[b + 1], q0), g.total_q);
        }
        nq = q1 - q0;
        kv_len = min(max(g.lens[b], 0), g.table_stride * g.P);
        c0 = ct * TILE;
        ncols = min(TILE, min(nq, g.max_q) * G - c0);
        kv_hi = max(pos_of(c0 + ncols - 1, G) + 1, 0);
        kv_lo = g.window > 0 ? min(max(pos_of(c0, G) - g.window + 1, 0), kv_hi) : 0;
        s_begin = kv_lo / STEP;
        steps = kv_hi > kv_lo ? (kv_hi + STEP - 1) / STEP - s_begin : 0;
        // a workgroup takes g.chunk steps whatever the sequence's length, so that
        // those of a batch of uneven lengths end together; more where the length
        // is past what the call named as the longest
        chunk = max(g.chunk, (steps + g.splits - 1) / g.splits);
        splits = max(1, (steps + chunk - 1) / chunk);
    }
    __device__ __forceinline__ int pos_of(int row, int G) const { return kv_len - nq + row / G; }
    // the steps of workgroup `split`: [first, end)
    __device__ __forceinline__ int first(int split) const {
        return s_begin + min(steps, split * chunk);
    }
};

// The rows of one workgroup's tile: partial sums joined in LDS, then written,
// or left in the workspace for kv4_reduce.hip.
template <int DT, int D>
struct AttnRows {
    static constexpr int kRow = D + 4;  // floats of a partial row: D sums, reference, sum of p, two unused
    const Kv4AttnArgs &g;
    int tile, splits, split, c0, q0, h, G;

    // (a sum of p that is not a number shows in the row)
    __device__ __forceinline__ static f32x4 quotient(f32x4 v, float sum, float ref) {
        sum = ref == kNoRef || fabsf(ref) < kFarRef ? sum : __builtin_nanf("");
        return sum == 0.0f ? (f32x4){0, 0, 0, 0} : v / sum;
    }
    __device__ __forceinline__ void put(int col, int d, f32x4 v) const {
        const int row = c0 + col, qi = row / G, hg = row - qi * G;
        *(uint2 *)((uint16_t *)g.out + ((size_t)(q0 + qi) * g.Hq + h * G + hg) * D + d) = quad_out_bits<DT>(v);
    }
    __device__ __forceinline__ float *row_of(int s, int col) const {
        return g.partials + (((size_t)tile * g.splits + s) * g.part_cols + col) * kRow;
    }
    // Rows col0 .. col0 + nc - 1 from NP partial rows each, in LDS at rows index(p, row - col0).
    template <int NP, typename Index>
    __device__ __forceinline__ void join(const float *lds, Index index, int col0, int nc) const {
        for (int i = threadIdx.x; i < nc * (D / 4); i += 64 * kAttnWaves) {
            const int col = i / (D / 4), d = 4 * (i % (D / 4));
            float rr = kNoRef, ll = 0.0f;
            f32x4 v = {0, 0, 0, 0};
#pragma unroll
            for (int p = 0; p < NP; ++p) rr = fmaxf(rr, lds[index(p, col) * kRow + D]);
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const float *row = lds + index(p, col) * kRow;
                const float a = __builtin_amdgcn_exp2f(row[D] - rr);
                v += a * *(const f32x4 *)(row + d);
                ll += a * row[D + 1];
            }
            if (splits == 1) {
                put(col0 + col, d, quotient(v, ll, rr));
            } else {
                float *row = row_of(split, col0 + col);
                *(f32x4 *)(row + d) = v;
                if (d == 0) *(f32x4 *)(row + D) = (f32x4){rr, ll, 0, 0};
            }
        }
    }
};

}  // namespace awq4
