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
// written once).  A lane holds 8 dimensions (16 bytes), D/8 lanes a head, so
// loads and q stores are whole cache lines, the abs-range of a head is a
// reduction over 8 or 16 neighbouring lanes and every lane packs one word.
// The partner of a half-split rotation is D/16 lanes away; it is read again
// (from the cache line that the neighbour just fetched) rather than moved
// between lanes, which would cost four shuffles.  Measured (32 heads over 8,
// D = 128, fp16): 8192 tokens 48 us, 3.8 TB/s of a copy's 4.9 (the cache's half of
// the writes is in pieces of 64 bytes and less); 64 tokens 3.8 us.
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

// One head's code words.  v: this lane's 8 values (16-bit patterns), LPH lanes
// a head.  Returns this lane's packed word and the head's meta word.
template <int DT, int LPH>
__device__ __forceinline__ uint32_t quantise_head(u32x4 v, uint32_t *meta) {
    // (largest key, largest complement of a key) of the lane, then of the head
    i16x2 top = {(int16_t)-32768, (int16_t)-32768}, bot = top;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint32_t key = order_key(v[p]);
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
        return 0u;
    }
    uint32_t w = 0;
    float z;
    auto code = [&](float q) { return (uint32_t)fminf(fmaxf(rintf(q) + z, 0.0f), 15.0f); };
    auto each = [&](auto divide) {
        z = fminf(rintf(divide(-lo)), 15.0f);
#pragma unroll
        for (int p = 0; p < 4; ++p) {  // columns 2p (nibble p) and 2p + 1 (nibble p + 4)
            w |= code(divide(act_bits_to_f32<DT>(v[p] & 0xFFFFu))) << (4 * p);
            w |= code(divide(act_bits_to_f32<DT>(v[p] >> 16))) << (4 * p + 16);
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

// One workgroup: one token's heads [256 / (D/8)] blockIdx.y ...; heads count
// queries first, then keys, then values.
template <int DT, int D>
__global__ __launch_bounds__(256) void kv4_append_kernel(Kv4AppendArgs g) {
    using L = Kv4Layout<D>;
    constexpr int LPH = D / 8;
    // 16 consecutive tokens to a die (workgroups go to the eight in turn): the
    // cache's lines hold words of 2 to 16 of them, and are written whole from one
    // die's cache (8192 tokens 50.4 -> 48.2 us; 4 or 64 tokens: 48.9, 48.1)
    const int i = blockIdx.x;
    const int t = i < (g.T & ~127) ? (i & ~127) + ((i & 7) << 4) + ((i >> 3) & 15) : i;
    const int head = blockIdx.y * (256 / LPH) + threadIdx.x / LPH;
    const int c = threadIdx.x % LPH, d = 8 * c;
    if (head >= g.Hq + 2 * g.Hkv) return;
    const int kind = head < g.Hq ? 0 : head < g.Hq + g.Hkv ? 1 : 2;
    const int h = head - (kind == 0 ? 0 : kind == 1 ? g.Hq : g.Hq + g.Hkv);
    const uint16_t *src = (const uint16_t *)(kind == 0 ? g.q : kind == 1 ? g.k : g.v) +
                          (size_t)t * (kind == 0 ? g.q_stride : kind == 1 ? g.k_stride : g.v_stride) + (size_t)h * D;
    const int64_t slot = g.slots[t];
    const bool stored = slot >= 0 && slot < g.num_pages * g.P;
    const int pos = g.rot > 0 ? g.positions[t] : 0;
    const bool placed = g.rot == 0 || (pos >= 0 && pos < g.max_pos);
    u32x4 v = *(const u32x4 *)(src + d);
    if (kind != 2 && d < g.rot) {
        if (!placed) {
            constexpr uint32_t nan2 = DT == DT_F16 ? 0x7E007E00u : 0x7FC07FC0u;
            v = (u32x4){nan2, nan2, nan2, nan2};
        } else if (g.interleaved) {
            // pairs (2i, 2i + 1): this lane's four pairs are angles d/2 .. d/2 + 3
            const float *cs = g.rope + (size_t)pos * g.rot + d / 2;
            const f32x4 co = *(const f32x4 *)cs, si = *(const f32x4 *)(cs + g.rot / 2);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const float a = act_bits_to_f32<DT>(v[p] & 0xFFFFu), b = act_bits_to_f32<DT>(v[p] >> 16);
                v[p] = (uint32_t)f32_to_out_bits(turn1(a, b, co[p], si[p]), DT) |
                       ((uint32_t)f32_to_out_bits(turn2(a, b, co[p], si[p]), DT) << 16);
            }
        } else {
            // pairs (i, i + rot/2): the other half's eight values
            const bool second = d >= g.rot / 2;
            const int i = second ? d - g.rot / 2 : d;
            const u32x4 o = *(const u32x4 *)(src + (second ? i : d + g.rot / 2));
            const float *cs = g.rope + (size_t)pos * g.rot + i;
            f32x4 co[2], si[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                co[u] = *(const f32x4 *)(cs + 4 * u);
                si[u] = *(const f32x4 *)(cs + g.rot / 2 + 4 * u);
            }
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                uint32_t bits = 0;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float me = act_bits_to_f32<DT>((v[p] >> (16 * e)) & 0xFFFFu);
                    const float it = act_bits_to_f32<DT>((o[p] >> (16 * e)) & 0xFFFFu);
                    const float cc = co[p >> 1][2 * (p & 1) + e], ss = si[p >> 1][2 * (p & 1) + e];
                    const float r = second ? turn2(it, me, cc, ss) : turn1(me, it, cc, ss);
                    bits |= (uint32_t)f32_to_out_bits(r, DT) << (16 * e);
                }
                v[p] = bits;
            }
        }
    }
    if (kind == 0) {
        *(u32x4 *)((uint16_t *)g.q_out + ((size_t)t * g.Hq + h) * D + d) = v;
        return;
    }
    uint32_t meta;
    const uint32_t w = quantise_head<DT, LPH>(v, &meta);
    if (!stored || !placed) return;
    const int64_t page = slot / g.P;
    const int in = (int)(slot - page * g.P);
    int32_t *base = g.cache + ((size_t)page * g.Hkv + h) * L::head_words(g.P);
    base[kind == 1 ? L::k_word(in, c) : L::v_word(g.P, in, c)] = (int32_t)w;
    if (c == 0) base[kind == 1 ? L::k_meta(g.P, in) : L::v_meta(g.P, in)] = (int32_t)meta;
}

template <int DT, int D>
static hipError_t launch_append(const Kv4AppendArgs &g, hipStream_t st) {
    constexpr int per = 256 / (D / 8);
    const int heads = g.Hq + 2 * g.Hkv;
    hipLaunchKernelGGL((kv4_append_kernel<DT, D>), dim3((unsigned)g.T, (unsigned)((heads + per - 1) / per)), dim3(256),
                       0, st, g);
    return hipGetLastError();
}

hipError_t launch_kv4_append(const Kv4AppendArgs &g, hipStream_t st) {
    if (g.D == 128)
        return g.dtype == DT_BF16 ? launch_append<DT_BF16, 128>(g, st) : launch_append<DT_F16, 128>(g, st);
    return g.dtype == DT_BF16 ? launch_append<DT_BF16, 64>(g, st) : launch_append<DT_F16, 64>(g, st);
}

}  // namespace awq4
