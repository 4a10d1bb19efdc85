// kv4_append.hip -- rotary positions on queries and keys, and keys and values
// quantised to 4 bits into the paged cache (layout: kv4.hpp).
//
// Rotation of the pair (x1, x2) with the position's cos c and sin s, fp32:
//   out1 = act(fl32(fl32(x1 c) - fl32(x2 s)))
//   out2 = act(fl32(fl32(x2 c) + fl32(x1 s)))
// (no fused multiply-adds, so that any fp32 program gets the same bits).
// Quantisation of one token and head x, after the rotation:
//   lo = min(0, min x), hi = max(0, max x), s = act(fl32(fl32(hi - lo) / 15))
//   z = clamp(rint(-lo / s), 0, 15), code = clamp(rint(x / s) + z, 0, 15)
// with correctly rounded fp32 quotients and rint to nearest even; s = 0 gives
// z = code = 0, and a head that holds a NaN or an infinity gives s = NaN, z =
// code = 0 (the attention over it is then NaN, as it would be unquantised).
//
// Bound: device memory (the 16-bit q, k, v read once, q and the packed words
// written once).  A lane holds two chunks of 8 dimensions, D/16 lanes a head: the
// partners of a half-split rotation, so that both come from one reading of the
// cosines and sines (16 fp32 numbers for 16 values; with a chunk a lane, its
// partner read beside it, twice that and half of the values again went through
// the CU's cache, and 8192 tokens took 48 us).  The abs-range of a head is a
// reduction over 4 or 8 neighbouring lanes, and every lane packs two words.
// Measured (32 heads over 8, D = 128, fp16): 8192 tokens 37 us, 4.9 TB/s, a
// copy's rate; 64 tokens 4.0 us.
#include "kv4.hpp"
#include "launch.hpp"

namespace awq4 {

typedef int16_t i16x2 __attribute__((ext_vector_type(2)));

// x / s correctly rounded to fp32, from r = RN(1 / s), for x and s of at most
// 11 bits (16-bit types): q0 = RN(x r) is off by less than two units, its
// remainder e is exact in one FMA (a multiple of a unit times s's last bit, of
// 13 bits at most), and q0 + e r is off by 2^-22 of a unit before its rounding,
// where x / s is never nearer than 2^-12 of one to a boundary between two
// results.  s in the normal range, and far enough from its ends that neither e
// nor q0 leaves it.
__device__ __forceinline__ float quotient(float x, float s, float r) {
    const float q0 = x * r;
    return __builtin_fmaf(__builtin_fmaf(-q0, s, x), r, q0);
}

__device__ __forceinline__ float turn1(float x1, float x2, float c, float s) {
#pragma clang fp contract(off)
    return x1 * c - x2 * s;
}
__device__ __forceinline__ float turn2(float x1, float x2, float c, float s) {
#pragma clang fp contract(off)
    return x2 * c + x1 * s;
}

// 16-bit patterns as integers in the order of the values (NaNs past the
// infinities of their sign), two at a time; its own inverse.
__device__ __forceinline__ uint32_t order_key(uint32_t b) {
    const i16x2 v = bit_as<i16x2>(b);
    return b ^ (bit_as<uint32_t>(v >> (int16_t)15) & 0x7FFF7FFFu);
}

// One head's code words.  v: this lane's two chunks of 8 values (16-bit
// patterns), LPH lanes a head.  Returns this lane's packed words and the head's
// meta word.
template <int DT, int LPH>
__device__ __forceinline__ u32x2 quantise_head(const u32x4 (&v)[2], uint32_t *meta) {
    // (largest key, largest complement of a key) of the lane, then of the head
    i16x2 top = {(int16_t)-32768, (int16_t)-32768}, bot = top;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const uint32_t key = order_key(v[n][p]);
            top = __builtin_elementwise_max(top, bit_as<i16x2>(key));
            bot = __builtin_elementwise_max(bot, bit_as<i16x2>(~key));
        }
    i16x2 both = {top[0] > top[1] ? top[0] : top[1], bot[0] > bot[1] ? bot[0] : bot[1]};
#pragma unroll
    for (int off = LPH / 2; off > 0; off >>= 1)
        both = __builtin_elementwise_max(both, bit_as<i16x2>(__shfl_xor(bit_as<int>(both), off, 64)));
    const uint32_t ends = order_key(bit_as<uint32_t>(both) ^ 0xFFFF0000u);  // patterns of the largest and the least
    constexpr uint32_t kInf = DT == DT_F16 ? 0x7C00u : 0x7F80u;
    const bool finite = (ends & 0x7FFFu) < kInf && ((ends >> 16) & 0x7FFFu) < kInf;
    const float hi = fmaxf(act_bits_to_f32<DT>(ends & 0xFFFFu), 0.0f);
    const float lo = fminf(act_bits_to_f32<DT>(ends >> 16), 0.0f);
    const uint16_t sb = f32_to_out_bits((hi - lo) / 15.0f, DT);
    const float s = act_bits_to_f32<DT>(sb);
    if (!finite || s == 0.0f) {
        *meta = finite ? 0u : kInf + 1u;  // a NaN, or zero
        return (u32x2){0, 0};
    }
    u32x2 w = {0, 0};
    float z;
    auto code = [&](float q) { return (uint32_t)fminf(fmaxf(rintf(q) + z, 0.0f), 15.0f); };
    auto each = [&](auto divide) {
        z = fminf(rintf(divide(-lo)), 15.0f);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int p = 0; p < 4; ++p) {  // columns 2p (nibble p) and 2p + 1 (nibble p + 4)
                w[n] |= code(divide(act_bits_to_f32<DT>(v[n][p] & 0xFFFFu))) << (4 * p);
                w[n] |= code(divide(act_bits_to_f32<DT>(v[n][p] >> 16))) << (4 * p + 16);
            }
    };
    // fp16 scales lie in 2^-24 .. 2^14; bf16 ones outside 2^-60 .. 2^120 divide
    if (DT == DT_F16 || (s > 0x1p-60f && s < 0x1p120f)) {
        const float r = 1.0f / s;
        each([&](float x) { return quotient(x, s, r); });
    } else {
        each([&](float x) { return x / s; });
    }
    *meta = (uint32_t)sb | ((uint32_t)z << 16);
    return w;
}

// One workgroup: one token's heads [blockDim.x / (D/16)] blockIdx.y ...; heads
// count queries first, then keys, then values.
template <int DT, int D>
__global__ __launch_bounds__(512) void kv4_append_kernel(Kv4AppendArgs g) {
    using L = Kv4Layout<D>;
    constexpr int LPH = D / 16;
    // 16 consecutive tokens to a die (workgroups go to the eight in turn): the
    // cache's lines hold words of 2 to 16 of them, and are written whole from one
    // die's cache (8192 tokens 50.4 -> 48.2 us; 4 or 64 tokens: 48.9, 48.1)
    const int i = blockIdx.x;
    const int t = i < (g.T & ~127) ? (i & ~127) + ((i & 7) << 4) + ((i >> 3) & 15) : i;
    const int head = blockIdx.y * (blockDim.x / LPH) + threadIdx.x / LPH;
    if (head >= g.Hq + 2 * g.Hkv) return;
    const int kind = head < g.Hq ? 0 : head < g.Hq + g.Hkv ? 1 : 2;
    const int h = head - (kind == 0 ? 0 : kind == 1 ? g.Hq : g.Hq + g.Hkv);
    const uint16_t *src = (const uint16_t *)(kind == 0 ? g.q : kind == 1 ? g.k : g.v) +
                          (size_t)t * (kind == 0 ? g.q_stride : kind == 1 ? g.k_stride : g.v_stride) + (size_t)h * D;
    // this lane's chunks of 8 dimensions, c and c + step: partners in a half-split
    // rotation; of the dimensions that do not turn, any two
    const int turning = g.rot / 16, lane = threadIdx.x % LPH;
    const bool turns = kind != 2 && lane < turning;
    const int c = lane < turning ? lane : turning + lane, step = lane < turning ? turning : LPH - turning;
    const int64_t slot = g.slots[t];
    const bool stored = slot >= 0 && slot < g.num_pages * g.P;
    const int pos = g.rot > 0 ? g.positions[t] : 0;
    const bool placed = g.rot == 0 || (pos >= 0 && pos < g.max_pos);
    u32x4 v[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) v[n] = *(const u32x4 *)(src + 8 * (c + n * step));
    if (turns && !placed) {
        constexpr uint32_t nan2 = DT == DT_F16 ? 0x7E007E00u : 0x7FC07FC0u;
        v[0] = v[1] = (u32x4){nan2, nan2, nan2, nan2};
    } else if (turns && g.interleaved) {
        // pairs (2i, 2i + 1): a chunk's four pairs are angles 4 chunk ..
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float *cs = g.rope + (size_t)pos * g.rot + 4 * (c + n * step);
            const f32x4 co = *(const f32x4 *)cs, si = *(const f32x4 *)(cs + g.rot / 2);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const float a = act_bits_to_f32<DT>(v[n][p] & 0xFFFFu), b = act_bits_to_f32<DT>(v[n][p] >> 16);
                v[n][p] = (uint32_t)f32_to_out_bits(turn1(a, b, co[p], si[p]), DT) |
                          ((uint32_t)f32_to_out_bits(turn2(a, b, co[p], si[p]), DT) << 16);
            }
        }
    } else if (turns) {
        // pairs (i, i + rot/2)
        const float *cs = g.rope + (size_t)pos * g.rot + 8 * c;
        f32x4 co[2], si[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            co[u] = *(const f32x4 *)(cs + 4 * u);
            si[u] = *(const f32x4 *)(cs + g.rot / 2 + 4 * u);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            uint32_t bits[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float a = act_bits_to_f32<DT>((v[0][p] >> (16 * e)) & 0xFFFFu);
                const float b = act_bits_to_f32<DT>((v[1][p] >> (16 * e)) & 0xFFFFu);
                const float cc = co[p >> 1][2 * (p & 1) + e], ss = si[p >> 1][2 * (p & 1) + e];
                bits[0] |= (uint32_t)f32_to_out_bits(turn1(a, b, cc, ss), DT) << (16 * e);
                bits[1] |= (uint32_t)f32_to_out_bits(turn2(a, b, cc, ss), DT) << (16 * e);
            }
            v[0][p] = bits[0];
            v[1][p] = bits[1];
        }
    }
    if (kind == 0) {
        uint16_t *out = (uint16_t *)g.q_out + ((size_t)t * g.Hq + h) * D;
#pragma unroll
        for (int n = 0; n < 2; ++n) *(u32x4 *)(out + 8 * (c + n * step)) = v[n];
        return;
    }
    uint32_t meta;
    const u32x2 w = quantise_head<DT, LPH>(v, &meta);
    if (!stored || !placed) return;
    const int64_t page = slot / g.P;
    const int in = (int)(slot - page * g.P);
    int32_t *base = g.cache + ((size_t)page * g.Hkv + h) * L::head_words(g.P);
#pragma unroll
    for (int n = 0; n < 2; ++n)
        base[kind == 1 ? L::k_word(in, c + n * step) : L::v_word(g.P, in, c + n * step)] = (int32_t)w[n];
    if (lane == 0) base[kind == 1 ? L::k_meta(g.P, in) : L::v_meta(g.P, in)] = (int32_t)meta;
}

template <int DT, int D>
static hipError_t launch_append(const Kv4AppendArgs &g, hipStream_t st) {
    constexpr int lph = D / 16, most = 512;
    const int lanes = (g.Hq + 2 * g.Hkv) * lph, parts = (lanes + most - 1) / most;
    // (whole waves, of about equal number in each part)
    const int threads = ((lanes + parts - 1) / parts + 63) / 64 * 64;
    hipLaunchKernelGGL((kv4_append_kernel<DT, D>), dim3((unsigned)g.T, (unsigned)parts), dim3(threads), 0, st, g);
    return hipGetLastError();
}

static hipError_t launch_part(const Kv4AppendArgs &g, hipStream_t st) {
    if (g.D == 128)
        return g.dtype == DT_BF16 ? launch_append<DT_BF16, 128>(g, st) : launch_append<DT_F16, 128>(g, st);
    return g.dtype == DT_BF16 ? launch_append<DT_BF16, 64>(g, st) : launch_append<DT_F16, 64>(g, st);
}

hipError_t launch_kv4_append(const Kv4AppendArgs &all, hipStream_t st) {
    for (int64_t t = 0; t < all.T; t += kLaunchRows) {
        auto tokens = [&](auto *p, int64_t bytes) { return p ? (decltype(p))((uintptr_t)p + t * bytes) : p; };
        Kv4AppendArgs g = all;
        g.T = all.T - t < kLaunchRows ? all.T - t : kLaunchRows;
        g.q = tokens(all.q, 2 * all.q_stride);
        g.k = tokens(all.k, 2 * all.k_stride);
        g.v = tokens(all.v, 2 * all.v_stride);
        g.positions = tokens(all.positions, 4);
        g.slots = tokens(all.slots, 8);
        g.q_out = tokens(all.q_out, (int64_t)2 * all.Hq * all.D);
        const hipError_t e = launch_part(g, st);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace awq4
