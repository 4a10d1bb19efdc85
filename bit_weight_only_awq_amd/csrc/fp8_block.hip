// fp8_block.hip -- 16-bit activations as E4M3 codes with one scale for each run
// of 128 values of a row:
//   s = fl32(max |x| / 448),  code = e4m3(clamp(fl32(x / s), -448, 448))
// A run lies in 16 lanes, 8 values each; the largest magnitude goes round the 16
// by moves inside the registers (as a whole number: the bit patterns of
// magnitudes order as they do, infinities and NaN last).  The quotient is the correctly rounded one without a
// divide per value (quant_ops.hpp): its r = 1 / s and the corrected quotient
// are correctly rounded for every normal s, whatever bits s has.  One
// launch, every value read once: bound by memory (4096 x 14336: 176 MB in 34.7 us, 5.1 TB/s, where a copy goes at
// 4.9; one row of 4096: 2.0 us).
#include "device.hpp"
#include "fp8_block.hpp"
#include "quant_ops.hpp"

namespace awq4 {

__device__ __forceinline__ uint32_t max16(uint32_t v) {
    auto dpp = [](uint32_t u, auto ctrl) {
        return (uint32_t)__builtin_amdgcn_mov_dpp((int)u, decltype(ctrl)::value, 0xF, 0xF, false);
    };
    v = max(v, dpp(v, std::integral_constant<int, 0xB1>{}));
    v = max(v, dpp(v, std::integral_constant<int, 0x4E>{}));
    v = max(v, dpp(v, std::integral_constant<int, 0x141>{}));
    return max(v, dpp(v, std::integral_constant<int, 0x140>{}));
}

template <int DT>
__global__ __launch_bounds__(256) void fp8_block_quant(const uint16_t *__restrict__ x, uint8_t *__restrict__ a,
                                                       float *__restrict__ s, int64_t runs, int K, int blocks) {
    const int64_t run = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    if (run >= runs) return;  // (whole groups of 16 lanes)
    const int64_t m = run / blocks;
    const int k = (int)(run - m * blocks) * kBlk + 8 * (threadIdx.x & 15);
    const bool have = k < K;
    const size_t at = (size_t)m * K + k;
    const u32x4 v = have ? *(const u32x4 *)(x + at) : (u32x4){0, 0, 0, 0};
    uint32_t mx = 0;
#pragma unroll
    for (int p = 0; p < 4; ++p) mx = max(mx, max(v[p] & 0x7FFFu, (v[p] >> 16) & 0x7FFFu));
    mx = max16(mx);
    const float sc = act_bits_to_f32<DT>(mx) / 448.0f;
    const Fp8Quotient<DT> fq(sc);
    u32x2 o = {0, 0};
    if (!fq.exact_divide) {
        o = (u32x2){fp8_codes4<DT>(fq, v[0], v[1]), fp8_codes4<DT>(fq, v[2], v[3])};
    } else if (sc > 0.0f && sc < __builtin_inff()) {
        // a scale below the normal numbers (bf16 only)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float q = act_bits_to_f32<DT>((v[e >> 1] >> (16 * (e & 1))) & 0xFFFFu) / sc;
            o[e >> 2] |= e4m3_code(fminf(fmaxf(q, -448.0f), 448.0f)) << (8 * (e & 3));
        }
    }
    if (have) *(u32x2 *)(a + at) = o;
    if ((threadIdx.x & 15) == 0) s[run] = sc;
}

hipError_t launch_fp8_block_quant(const void *x, uint8_t *a, float *s, int64_t M, int64_t K, int dtype,
                                  hipStream_t st) {
    const int64_t blocks = (K + kBlk - 1) / kBlk;
    // (less than 2^32 threads a launch: 2^24 workgroups of 256 are 2^28 runs)
    const int64_t rows = ((int64_t(1) << 27) / blocks);
    for (int64_t m = 0; m < M; m += rows) {
        const int64_t runs = (M - m < rows ? M - m : rows) * blocks;
        const dim3 grid((unsigned)((runs + 15) / 16));
        const uint16_t *xm = (const uint16_t *)x + m * K;
        if (dtype == DT_BF16)
            hipLaunchKernelGGL(fp8_block_quant<DT_BF16>, grid, dim3(256), 0, st, xm, a + m * K, s + m * blocks, runs,
                               (int)K, (int)blocks);
        else
            hipLaunchKernelGGL(fp8_block_quant<DT_F16>, grid, dim3(256), 0, st, xm, a + m * K, s + m * blocks, runs,
                               (int)K, (int)blocks);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace awq4
