// quant_ops.hpp -- per-token activation quantisation primitives, shared by the
// quantisers (w4a8.hip, w4a8_fp8.hip) and the RMS norm that writes 8-bit codes
// (norm.hip): the int8 and E4M3 codes of 16-bit values for a row's scale.
#pragma once

#include "device.hpp"

namespace awq4 {

// Rounding an fp32 value to the activation type (nearest even) and back.
template <int DT>
__device__ __forceinline__ float round_to_act(float v) {
    return DT == DT_F16 ? (float)(f16)v : (float)(__bf16)v;
}

// ---------------------------------------------------------------------------
// int8 codes of 8 fp16 or bf16 values (one 16-byte chunk) for the scale s,
// given r ~ 1/s: round half to even of x / s, clamped to int8, without a
// divide.  For x and s of one 16-bit type the exact quotient is a half-integer
// or at least 2^-12 (fp16) / 2^-9 (bf16) from one, and x * r (r within a few
// ulps of 1/s) stays within 2^-15 of it.
// One FMA adds 1536, which rounds x * r to a multiple of 2^-13 (the fp32
// spacing in [1024, 2048)): exact ties land on the half-integer, every other
// quotient stays on its own side of it.  The clamp is taken in that shifted
// range; adding 1.5 * 2^23 - 1536 then rounds to an integer (half to even)
// held in the low mantissa bits, so the low byte of the sum's bits is the
// int8 code.  Checked exhaustively against the correctly rounded fp32 divide
// for every reachable s (bf16: every s >= 2^-126, whose reciprocal is a normal
// fp32 value; smaller scales take the divide), every x and reciprocals up to
// 3 ulps off.
template <int DT>
__device__ __forceinline__ u32x2 quant8(u32x4 v, float r) {
    uint32_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float f = act_bits_to_f32<DT>((v[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
        const float t = __builtin_amdgcn_fmed3f(__builtin_fmaf(f, r, 1536.0f), 1536.0f - 128.0f, 1536.0f + 127.0f);
        b[e] = bit_as<uint32_t>(t + (12582912.0f - 1536.0f));
    }
    u32x2 o;
#pragma unroll
    for (int w = 0; w < 2; ++w)  // low bytes of b[4w .. 4w+3]
        o[w] = perm_b32(b[4 * w + 1], b[4 * w], 0x0C0C0400u) | perm_b32(b[4 * w + 3], b[4 * w + 2], 0x04000C0Cu);
    return o;
}

// The same codes through the correctly rounded fp32 divide (bf16 scales
// below 2^-126, whose reciprocal is not a normal fp32 value).
template <int DT>
__device__ __forceinline__ u32x2 quant8_div(u32x4 v, float s) {
    u32x2 o = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t h = (v[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
        const float qf = fminf(fmaxf(rintf(act_bits_to_f32<DT>(h) / s), -128.0f), 127.0f);
        o[e >> 2] |= ((uint32_t)(int32_t)qf & 0xFFu) << (8 * (e & 3));
    }
    return o;
}

// ---------------------------------------------------------------------------
// E4M3 code of |q| <= 448 (not NaN), round to nearest, ties to even.
__device__ __forceinline__ uint32_t e4m3_code(float q) {
    const uint32_t u = bit_as<uint32_t>(q);
    const uint32_t sign = (u >> 24) & 0x80u;
    const uint32_t a = u & 0x7FFFFFFFu;
    uint32_t code;
    if (a < 0x3C800000u) {
        // below 2^-6: multiples of 2^-9 (the scaling by 512 is exact)
        code = (uint32_t)__builtin_rintf(bit_as<float>(a) * 512.0f);
    } else {
        // round the fp32 significand to 3 bits (nearest even), then rebias
        // the exponent from 127 to 7; a carry moves into the exponent
        const uint32_t r = (a + 0x7FFFFu + ((a >> 20) & 1u)) >> 20;
        code = r - ((127u - 7u) << 3);
    }
    return sign | code;
}

// Value of an E4M3 code in units of 2^-9 (an exact integer, |v| <= 229376).
__device__ __forceinline__ int32_t e4m3_units(uint32_t c) {
    const int32_t e = (c >> 3) & 15, m = c & 7;
    const int32_t v = e == 0 ? m : (8 + m) << (e - 1);
    return (c & 0x80u) ? -v : v;
}

// ---------------------------------------------------------------------------
// The quotient x / s without a divide per value.  Per row: r = RN(1 / s') by
// one divide; per value q0 = RN(x' r), e = x' - q0 s' (exact, one FMA) and
// q = RN(q0 + e r), Markstein's correction, which is the correctly rounded
// quotient when nothing underflows; x' and s' are x and s times 2^64 on bf16
// rows with s < 2^-60 (exact, the same quotient), so that every x whose
// quotient can reach the smallest E4M3 subnormal stays far above the range
// where e would round.  Checked on the host for every scale the quantiser can
// produce and every fp16 / bf16 value it can meet: the E4M3 code of the
// clamped q equals that of the clamped correctly rounded quotient in every
// case.  Rows with s = 0, s below 2^-126 (bf16 only) or s not finite take
// the divide.
template <int DT>
struct Fp8Quotient {
    float sc, ss, r;
    bool exact_divide;
    __device__ __forceinline__ explicit Fp8Quotient(float s) {
        sc = (DT == DT_BF16 && s < 0x1p-60f) ? 0x1p64f : 1.0f;
        ss = s * sc;
        exact_divide = !(s >= 0x1p-126f && s <= 3.4028234663852886e38f);
        r = exact_divide ? 0.0f : 1.0f / ss;
    }
    // clamp(x / s, +-448) for exact_divide == false.  The sign is x's: the
    // correction can turn a zero quotient's sign (-0 + 0 = +0), and the E4M3
    // code keeps it.
    __device__ __forceinline__ float q(float x) const {
        const float xs = DT == DT_BF16 ? x * sc : x;
        const float q0 = xs * r;
        const float e = __builtin_fmaf(-q0, ss, xs);
        return __builtin_amdgcn_fmed3f(__builtin_copysignf(__builtin_fmaf(e, r, q0), x), -448.0f, 448.0f);
    }
};

// E4M3 codes of the clamped quotients of four 16-bit activation patterns
// (h01: values 0, 1 in its halves; h23: values 2, 3), one byte each, by the
// matrix-core generation's fp32 -> OCP E4M3 conversion (round to nearest
// even; the same code as e4m3_code for every |q| <= 448, both signs,
// subnormals included -- checked on the device over all such fp32 values).
template <int DT>
__device__ __forceinline__ uint32_t fp8_codes4(const Fp8Quotient<DT> &f, uint32_t h01, uint32_t h23) {
    const float q0 = f.q(act_bits_to_f32<DT>(h01 & 0xFFFFu)), q1 = f.q(act_bits_to_f32<DT>(h01 >> 16));
    const float q2 = f.q(act_bits_to_f32<DT>(h23 & 0xFFFFu)), q3 = f.q(act_bits_to_f32<DT>(h23 >> 16));
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q0, q1, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q2, q3, lo, true);
}

// Sum of the values of eight E4M3 codes (one a byte of lo, hi), in units of
// 2^-9, through the hardware's fp8 -> fp32 decode (the same OCP E4M3 format
// as the encode above).  Exact: every value is a multiple of 2^-9 of
// magnitude at most 448, so every partial sum of the eight is a multiple of
// 2^-9 below 2^24 units and fp32 holds it.
__device__ __forceinline__ int32_t e4m3_units8(uint32_t lo, uint32_t hi) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)lo, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)lo, true);
    const f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8((int)hi, false), d = __builtin_amdgcn_cvt_pk_f32_fp8((int)hi, true);
    const float v = ((a[0] + a[1]) + (b[0] + b[1])) + ((c[0] + c[1]) + (d[0] + d[1]));
    return (int32_t)(v * 512.0f);
}

}  // namespace awq4
