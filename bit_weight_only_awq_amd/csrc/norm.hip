// norm.hip -- residual addition, root-mean-square norm and per-token 8-bit
// quantisation in one pass over the rows: the activations that a W4A8 or
// INT4-FP8 layer takes, straight from the hidden state.
//
//   h = act(fl32(x + r))                       (no residual: h = x)
//   v = fl32(sum_k h^2 / K + eps)              the sum and the mean in binary64
//   q = fl32(1 / fl32(sqrt(v)))
//   y = act(fl32(fl32(h q) w))
// then the codes and scales that the quantisers (w4a8.hip, w4a8_fp8.hip) give
// of y, bit for bit.  Every rounding above is part of the definition; only the
// order in which the squares are summed is not.  It depends on K alone, so a
// row's results are the same in every launch, and most sums' bits all fit in
// binary64, so that no order matters: another's error (2^-53 an addition) changes
// v's rounding to binary32 in fewer than one row of 10^6.
//
// Bound: device memory.  A row is read once (x, r, w), held in registers as h
// and then y, and written once (h, codes, s1, y if asked for): 7 bytes a value
// with the residual against 13 in two launches (norm, then quantiser).  4096
// rows of 4096 values, fp16, int8 codes: 21.5 us, 5.5 TB/s.  One row takes 2.6 us:
// a memory round trip and two sums over the workgroup.
#include "device.hpp"
#include "launch.hpp"
#include "quant_ops.hpp"

namespace awq4 {

enum { NORM_PLAIN = 0, NORM_INT8 = 1, NORM_FP8 = 2 };

// Sum over the 64 lanes of a wave, the same bits in every lane.
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, 64));
    return v;
}

// Two fp32 values as a pair of the activation type.  The values are made
// opaque first: the compiler otherwise merges the operation before the
// conversion into one that rounds once, to the 16-bit type (v_fma_mixlo_f16),
// and the definition rounds to binary32 in between.
template <int DT>
__device__ __forceinline__ uint32_t pair_act(float lo, float hi) {
    asm("" : "+v"(lo), "+v"(hi));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const f32x2 v = {lo, hi};
    if (DT == DT_F16) return bit_as<uint32_t>(__builtin_convertvector(v, f16x2));
    return bit_as<uint32_t>(__builtin_convertvector(v, bf16x2));
}
template <int DT>
__device__ __forceinline__ uint16_t one_act(float v) {
    asm("" : "+v"(v));
    return f32_to_out_bits(v, DT);
}

template <int DT>
__device__ __forceinline__ uint32_t add_act(uint32_t a, uint32_t b) {  // two values
    return pair_act<DT>(act_bits_to_f32<DT>(a & 0xFFFFu) + act_bits_to_f32<DT>(b & 0xFFFFu),
                        act_bits_to_f32<DT>(a >> 16) + act_bits_to_f32<DT>(b >> 16));
}
template <int DT>
__device__ __forceinline__ double square2(uint32_t a) {
    const double lo = act_bits_to_f32<DT>(a & 0xFFFFu), hi = act_bits_to_f32<DT>(a >> 16);
    return __builtin_fma(lo, lo, hi * hi);
}
template <int DT>
__device__ __forceinline__ uint32_t scale_act(uint32_t h, uint32_t w, float q) {
    return pair_act<DT>(act_bits_to_f32<DT>(h & 0xFFFFu) * q * act_bits_to_f32<DT>(w & 0xFFFFu),
                        act_bits_to_f32<DT>(h >> 16) * q * act_bits_to_f32<DT>(w >> 16));
}
// The row's factor from its sum of squares.  A division, not a product with
// 1 / K: its rounding error would reach v where the mean lies next to the middle
// between two binary32 numbers.
__device__ __forceinline__ float rms_factor(double sum, int K, float eps) {
    const float v = (float)(sum / (double)K + (double)eps);
    return 1.0f / __builtin_sqrtf(v);
}

// Register-resident form: one workgroup of T threads per row, each thread
// holding NV chunks of 8 values (K % 8 == 0, K <= 8 NV T).  The row's weights
// are loaded with x, before the first reduction, so that one memory round trip
// covers all inputs.  x may be y, and r may be h_out: a row's values are all
// in registers before the first store.
template <int DT, int OUT, int NV, int T>
__global__ __launch_bounds__(T) void rmsnorm_rows(const uint16_t *x, const uint16_t *r,
                                                  const uint16_t *__restrict__ w, uint16_t *h_out, uint16_t *y,
                                                  uint8_t *__restrict__ a, float *__restrict__ s1,
                                                  float *__restrict__ asum, int K, float eps) {
    constexpr int W = T / 64;
    __shared__ double wsum[W];
    __shared__ uint32_t wmax[W];
    __shared__ long long wcode[W];
    const int m = blockIdx.x, wave = threadIdx.x >> 6;
    const bool leader = (threadIdx.x & 63) == 0;
    const size_t at = (size_t)m * K;
    u32x4 v[NV], wt[NV];
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int k = 8 * (threadIdx.x + i * T);
        const bool in = k < K;
        v[i] = in ? *(const u32x4 *)(x + at + k) : (u32x4){0, 0, 0, 0};
        wt[i] = in ? *(const u32x4 *)(w + k) : (u32x4){0, 0, 0, 0};
        if (r && in) {
            const u32x4 rv = *(const u32x4 *)(r + at + k);
#pragma unroll
            for (int p = 0; p < 4; ++p) v[i][p] = add_act<DT>(v[i][p], rv[p]);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int k = 8 * (threadIdx.x + i * T);
#pragma unroll
        for (int p = 0; p < 4; ++p) sum += square2<DT>(v[i][p]);
        if (h_out && k < K) *(u32x4 *)(h_out + at + k) = v[i];
    }
    sum = wave_sum(sum);
    if (leader) wsum[wave] = sum;
    __syncthreads();
    sum = wsum[0];
#pragma unroll
    for (int i = 1; i < W; ++i) sum += wsum[i];
    const float q = rms_factor(sum, K, eps);
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int k = 8 * (threadIdx.x + i * T);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            v[i][p] = scale_act<DT>(v[i][p], wt[i][p], q);
            mx = max(mx, max(v[i][p] & 0x7FFFu, (v[i][p] >> 16) & 0x7FFFu));
        }
        if (y && k < K) *(u32x4 *)(y + at + k) = v[i];
    }
    if (OUT == NORM_PLAIN) return;
    mx = wave_max(mx);
    if (leader) wmax[wave] = mx;
    __syncthreads();
    mx = wmax[0];
#pragma unroll
    for (int i = 1; i < W; ++i) mx = max(mx, wmax[i]);
    const float amax = act_bits_to_f32<DT>(mx);
    if (OUT == NORM_INT8) {
        const float s = round_to_act<DT>(amax / 127.0f);
        if (threadIdx.x == 0) s1[m] = s;
        const float rs = __builtin_amdgcn_rcpf(s);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = 8 * (threadIdx.x + i * T);
            if (k >= K) break;
            u32x2 o = {0, 0};
            if (s != 0.0f) o = (DT == DT_F16 || s >= 0x1p-126f) ? quant8<DT>(v[i], rs) : quant8_div<DT>(v[i], s);
            *(u32x2 *)(a + at + k) = o;
        }
    } else {
        const float s = round_to_act<DT>(amax / 448.0f);
        const Fp8Quotient<DT> fq(s);
        long long units = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = 8 * (threadIdx.x + i * T);
            if (k >= K) break;
            u32x2 o = {0, 0};
            if (!fq.exact_divide) {
                o = (u32x2){fp8_codes4<DT>(fq, v[i][0], v[i][1]), fp8_codes4<DT>(fq, v[i][2], v[i][3])};
                units += e4m3_units8(o[0], o[1]);
            } else if (s != 0.0f) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float f = act_bits_to_f32<DT>((v[i][e >> 1] >> (16 * (e & 1))) & 0xFFFFu) / s;
                    const uint32_t c = e4m3_code(fminf(fmaxf(f, -448.0f), 448.0f));
                    units += e4m3_units(c);
                    o[e >> 2] |= c << (8 * (e & 3));
                }
            }
            *(u32x2 *)(a + at + k) = o;
        }
        units = wave_sum(units);
        if (leader) wcode[wave] = units;
        __syncthreads();
        if (threadIdx.x == 0) {
            units = 0;
#pragma unroll
            for (int i = 0; i < W; ++i) units += wcode[i];
            s1[m] = s;
            asum[m] = (float)units * 0x1p-9f;  // one rounding (int64 -> fp32), then an exact power of two
        }
    }
}

// General form (any K): one workgroup of 256 threads per row, a value at a
// time, three passes (sum of squares, abs-max, codes); 1024 rows of 4097 values,
// fp16, int8, 22.5 us where 4096 in registers take 8.6.  Each thread reads in
// the later passes only what it wrote or left unchanged itself: h from h_out
// where there is a residual, y from y where it is asked for.
template <int DT, int OUT>
__global__ __launch_bounds__(256) void rmsnorm_any(const uint16_t *x, const uint16_t *r, const uint16_t *w,
                                                   uint16_t *h_out, uint16_t *y, uint8_t *a, float *s1, float *asum,
                                                   int K, float eps) {
    __shared__ double wsum[4];
    __shared__ uint32_t wmax[4];
    __shared__ long long wcode[4];
    const int m = blockIdx.x, wave = threadIdx.x >> 6;
    const bool leader = (threadIdx.x & 63) == 0;
    const size_t at = (size_t)m * K;
    double sum = 0.0;
    for (int k = threadIdx.x; k < K; k += 256) {
        float h = act_bits_to_f32<DT>(x[at + k]);
        if (r) {
            const uint16_t b = one_act<DT>(h + act_bits_to_f32<DT>(r[at + k]));
            h_out[at + k] = b;
            h = act_bits_to_f32<DT>(b);
        }
        sum = __builtin_fma((double)h, (double)h, sum);
    }
    sum = wave_sum(sum);
    if (leader) wsum[wave] = sum;
    __syncthreads();
    sum = (wsum[0] + wsum[1]) + (wsum[2] + wsum[3]);
    const float q = rms_factor(sum, K, eps);
    const uint16_t *h = r ? h_out : x;
    auto value = [&](int k) -> uint32_t {
        return one_act<DT>(act_bits_to_f32<DT>(h[at + k]) * q * act_bits_to_f32<DT>(w[k]));
    };
    uint32_t mx = 0;
    for (int k = threadIdx.x; k < K; k += 256) {
        const uint32_t b = value(k);
        mx = max(mx, b & 0x7FFFu);
        if (y) y[at + k] = (uint16_t)b;
    }
    if (OUT == NORM_PLAIN) return;
    mx = wave_max(mx);
    if (leader) wmax[wave] = mx;
    __syncthreads();
    mx = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
    const float s = round_to_act<DT>(act_bits_to_f32<DT>(mx) / (OUT == NORM_INT8 ? 127.0f : 448.0f));
    long long units = 0;
    for (int k = threadIdx.x; k < K; k += 256) {
        const float f = act_bits_to_f32<DT>(y ? (uint32_t)y[at + k] : value(k)) / s;
        if (OUT == NORM_INT8) {
            a[at + k] = s == 0.0f ? 0 : (uint8_t)(int8_t)fminf(fmaxf(rintf(f), -128.0f), 127.0f);
        } else {
            const uint32_t c = s == 0.0f ? 0u : e4m3_code(fminf(fmaxf(f, -448.0f), 448.0f));
            units += e4m3_units(c);
            a[at + k] = (uint8_t)c;
        }
    }
    if (threadIdx.x == 0) s1[m] = s;
    if (OUT == NORM_FP8) {
        units = wave_sum(units);
        if (leader) wcode[wave] = units;
        __syncthreads();
        if (threadIdx.x == 0) asum[m] = (float)(wcode[0] + wcode[1] + wcode[2] + wcode[3]) * 0x1p-9f;
    }
}

template <int DT, int OUT, int NV, int T>
static hipError_t launch_rows(const NormArgs &n, hipStream_t st) {
    hipLaunchKernelGGL((rmsnorm_rows<DT, OUT, NV, T>), dim3((unsigned)n.M), dim3(T), 0, st, (const uint16_t *)n.x,
                       (const uint16_t *)n.residual, (const uint16_t *)n.weight, (uint16_t *)n.residual_out,
                       (uint16_t *)n.y, (uint8_t *)n.a, n.s1, n.asum, (int)n.K, n.eps);
    return hipGetLastError();
}

// Threads for a row: 8 values each up to 512 threads, then two chunks each up
// to 8192 values, then 1024 threads.  Both sides, with a residual, in us:
//   8192 values, bf16, fp8 codes   rows     1    64   300   777  2048  4096
//     512 threads                         5.0   5.4   8.2  14.6  24.7  45.8
//     256                                 5.9   6.5   8.7  14.0  24.4  49.4
//   5120 values, fp16, int8 codes
//     512                                 4.0   4.4   5.7  10.5  17.3  32.0
//     256                                 4.7   5.1   6.1  10.1  17.6  32.4
//   14336 values, bf16, fp8 codes  rows     1   300   777  2048
//     1024                                6.2  12.9  22.0  45.6
//     512                                 6.3  12.3  22.2  48.2
// (777 rows of 8192 in 1024 threads 15.4; 4096 rows of 4096, fp16, int8: 512
// threads 21.5, 256 22.8.)
template <int DT, int OUT>
static hipError_t launch_norm(const NormArgs &n, hipStream_t st) {
    if (n.K % 8 == 0 && n.K <= 8 * 1024 * 4) {
        if (n.K <= 8 * 128) return launch_rows<DT, OUT, 1, 128>(n, st);
        if (n.K <= 8 * 256) return launch_rows<DT, OUT, 1, 256>(n, st);
        if (n.K <= 8 * 512) return launch_rows<DT, OUT, 1, 512>(n, st);
        if (n.K <= 8 * 1024) return launch_rows<DT, OUT, 2, 512>(n, st);
        if (n.K <= 8 * 1024 * 2) return launch_rows<DT, OUT, 2, 1024>(n, st);
        return launch_rows<DT, OUT, 4, 1024>(n, st);
    }
    hipLaunchKernelGGL((rmsnorm_any<DT, OUT>), dim3((unsigned)n.M), dim3(256), 0, st, (const uint16_t *)n.x,
                       (const uint16_t *)n.residual, (const uint16_t *)n.weight, (uint16_t *)n.residual_out,
                       (uint16_t *)n.y, (uint8_t *)n.a, n.s1, n.asum, (int)n.K, n.eps);
    return hipGetLastError();
}

template <int DT>
static hipError_t launch_norm_dt(const NormArgs &n, hipStream_t st) {
    if (!n.a) return launch_norm<DT, NORM_PLAIN>(n, st);
    return n.asum ? launch_norm<DT, NORM_FP8>(n, st) : launch_norm<DT, NORM_INT8>(n, st);
}

hipError_t launch_rmsnorm(const NormArgs &all, hipStream_t st) {
    for (int64_t m = 0; m < all.M; m += kLaunchRows) {
        auto rows = [&](auto *p, int64_t bytes) { return p ? (decltype(p))((uintptr_t)p + m * bytes) : p; };
        NormArgs n = all;
        n.M = all.M - m < kLaunchRows ? all.M - m : kLaunchRows;
        n.x = rows(all.x, 2 * all.K);
        n.residual = rows(all.residual, 2 * all.K);
        n.residual_out = rows(all.residual_out, 2 * all.K);
        n.y = rows(all.y, 2 * all.K);
        n.a = rows(all.a, all.K);
        n.s1 = rows(all.s1, 4);
        n.asum = rows(all.asum, 4);
        const hipError_t e = n.dtype == DT_BF16 ? launch_norm_dt<DT_BF16>(n, st) : launch_norm_dt<DT_F16>(n, st);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace awq4
