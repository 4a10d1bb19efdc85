// split_sum.hip -- the K splits' sums of a product through LDS tiles (grouped by expert, or block-scaled E4M3)
// [S][M][N] in fp32, added in split order, written and cleared; one thread a quad of outputs.  Bound by memory: S x 4
// bytes an output read, S x 4 + 2 written.  Rows before the first expert's and behind the last's (offsets: the one and
// the other) are not written, but cleared like the others: offsets that are no plan leave nothing behind either.
#include "device.hpp"
#include "launch.hpp"

namespace awq4 {

template <int DT>
__global__ __launch_bounds__(256) void split_sum(f32x4 *__restrict__ part, uint16_t *__restrict__ y,
                                                 const int32_t *__restrict__ offsets, int E, int64_t quads, int N, int S) {
    const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (q >= quads) return;
    const int64_t row = q / (N / 4);
    const bool live = !offsets || (row >= offsets[0] && row < offsets[E]);
    f32x4 v = (f32x4){0.f, 0.f, 0.f, 0.f};
    constexpr int kB = 4;
    for (int s0 = 0; s0 < S; s0 += kB) {
        f32x4 b[kB];
#pragma unroll
        for (int i = 0; i < kB; ++i) b[i] = s0 + i < S ? part[q + (s0 + i) * quads] : (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kB; ++i)
            if (s0 + i < S) v += b[i];
    }
    if (live) *(uint2 *)(y + 4 * q) = quad_out_bits<DT>(v);
    for (int s = 0; s < S; ++s) part[q + s * quads] = (f32x4){0.f, 0.f, 0.f, 0.f};
}

hipError_t launch_split_sum(void *part, void *y, const int32_t *offsets, int E, int64_t M, int64_t N, int S, int dtype,
                            hipStream_t st) {
    const int64_t quads = M * N / 4;
    const dim3 grid((unsigned)((quads + 255) / 256));
    if (dtype == DT_BF16)
        hipLaunchKernelGGL(split_sum<DT_BF16>, grid, dim3(256), 0, st, (f32x4 *)part, (uint16_t *)y, offsets, E, quads,
                           (int)N, S);
    else
        hipLaunchKernelGGL(split_sum<DT_F16>, grid, dim3(256), 0, st, (f32x4 *)part, (uint16_t *)y, offsets, E, quads,
                           (int)N, S);
    return hipGetLastError();
}

}  // namespace awq4
