// kv4_reduce.hip -- the sums of an attention call's workgroups, where several
// share a sequence: a kernel after the attention kernel (any but that for tiles
// of 32 rows, which fill the device by themselves) adds them, writes the rows
// and clears the workspace.  (Added in the attention
// kernels by the last workgroup to arrive, through the device's coherence point,
// they took longer at every number of splits tried from 2 on: 4 x 24 rows over
// 1024 tokens 18.7 us against 16.6, 4 x 256 rows 68 against 46; a single row
// about the same.)
//
// Bound: latency, and the volume of the partial sums (4 (D + 4) bytes a row
// and workgroup, written, read and cleared).  A row's D/4 quads lie side by
// side in a workgroup of 256 threads.  Up to kFew splits, a thread adds all of
// a row's quad, and the workgroup takes as many rows as fit; more, and the
// remaining factor of the threads shares one row's splits, every load in
// flight at once, the sums joined in LDS in the splits' order.  (One row a
// workgroup at 2 splits of 4 x 1024 rows: 141 us with the attention, 46 as it is.)
#include "kv4_ops.hpp"

namespace awq4 {

constexpr int kFew = 8;

// The tile and the rows of workgroup (blockIdx.x, blockIdx.y), in the attention
// kernels' order of tiles.
template <int DT, int D, int TILE, int STEP>
struct ReduceTile {
    int h, b, G;
    const Kv4Span<TILE, STEP> span;
    const AttnRows<DT, D> out;
    __device__ __forceinline__ static int col_tile(const Kv4AttnArgs &g) {
        return TILE == 256 ? blockIdx.x / (g.B * g.Hkv) : blockIdx.x % g.col_tiles;
    }
    __device__ __forceinline__ static int head(const Kv4AttnArgs &g) {
        return TILE == 256 ? blockIdx.x % (g.B * g.Hkv) : blockIdx.x / g.col_tiles;
    }
    __device__ __forceinline__ explicit ReduceTile(const Kv4AttnArgs &g)
        : h(head(g) % g.Hkv), b(head(g) / g.Hkv), G(g.Hq / g.Hkv), span(g, b, col_tile(g), G),
          out{g, (int)blockIdx.x, span.splits, 0, span.c0, span.q0, h, G} {}
};

template <int DT, int D, int TILE, int STEP>
__global__ __launch_bounds__(256) void kv4_reduce_few_kernel(Kv4AttnArgs g) {
    constexpr int Q = D / 4, ROWS = 256 / Q;
    const int q = threadIdx.x % Q, col = blockIdx.y * ROWS + threadIdx.x / Q;
    const ReduceTile<DT, D, TILE, STEP> t(g);
    const int splits = t.span.splits;
    if (col >= t.span.ncols || splits == 1) return;
    f32x4 w[kFew];
    f32x2 rl[kFew];
#pragma unroll
    for (int s = 0; s < kFew; ++s) {
        const bool in = s < splits;
        const float *row = t.out.row_of(in ? s : 0, col);
        w[s] = in ? *(const f32x4 *)(row + 4 * q) : (f32x4){0, 0, 0, 0};
        rl[s] = in ? *(const f32x2 *)(row + D) : (f32x2){kNoRef, 0.0f};
    }
    float rr = kNoRef, ll = 0.0f;
#pragma unroll
    for (int s = 0; s < kFew; ++s) rr = fmaxf(rr, rl[s][0]);
    f32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < kFew; ++s) {
        const float a = __builtin_amdgcn_exp2f(rl[s][0] - rr);
        v += a * w[s];
        ll += a * rl[s][1];
    }
    t.out.put(col, 4 * q, AttnRows<DT, D>::quotient(v, ll, rr));
    // (the threads of a row are of one wave, so all of them have read its references)
    for (int s = 0; s < splits; ++s) {
        *(f32x4 *)(t.out.row_of(s, col) + 4 * q) = (f32x4){0, 0, 0, 0};
        if (q == 0) *(f32x4 *)(t.out.row_of(s, col) + D) = (f32x4){0, 0, 0, 0};
    }
}

template <int DT, int D, int TILE, int STEP>
__global__ __launch_bounds__(256) void kv4_reduce_kernel(Kv4AttnArgs g) {
    constexpr int Q = D / 4, GROUPS = 256 / Q, SHARE = (kKv4MaxSplits + GROUPS - 1) / GROUPS;
    __shared__ f32x4 lds_v[GROUPS][Q];
    __shared__ float lds_r[GROUPS], lds_l[GROUPS];
    const int col = blockIdx.y, q = threadIdx.x % Q, group = threadIdx.x / Q;
    const ReduceTile<DT, D, TILE, STEP> t(g);
    const auto &span = t.span;
    const auto &out = t.out;
    if (col >= span.ncols || span.splits == 1) return;
    f32x4 w[SHARE];
    float r[SHARE], l[SHARE], rr = kNoRef;
#pragma unroll
    for (int k = 0; k < SHARE; ++k) {
        const int s = group + GROUPS * k;
        const bool in = s < span.splits;
        const float *row = out.row_of(in ? s : 0, col);
        w[k] = in ? *(const f32x4 *)(row + 4 * q) : (f32x4){0, 0, 0, 0};
        const f32x2 rl = in ? *(const f32x2 *)(row + D) : (f32x2){kNoRef, 0.0f};
        r[k] = rl[0];
        l[k] = rl[1];
    }
#pragma unroll
    for (int k = 0; k < SHARE; ++k) rr = fmaxf(rr, r[k]);
    if (q == 0) lds_r[group] = rr;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) rr = fmaxf(rr, lds_r[i]);
    f32x4 v = {0, 0, 0, 0};
    float ll = 0.0f;
#pragma unroll
    for (int k = 0; k < SHARE; ++k) {
        const float a = __builtin_amdgcn_exp2f(r[k] - rr);
        v += a * w[k];
        ll += a * l[k];
    }
    lds_v[group][q] = v;
    if (q == 0) lds_l[group] = ll;
    __syncthreads();
    if (group == 0) {
        v = (f32x4){0, 0, 0, 0};
        ll = 0.0f;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            v += lds_v[i][q];
            ll += lds_l[i];
        }
        out.put(col, 4 * q, AttnRows<DT, D>::quotient(v, ll, rr));
    }
    for (int s = group; s < span.splits; s += GROUPS) {
        *(f32x4 *)(out.row_of(s, col) + 4 * q) = (f32x4){0, 0, 0, 0};
        if (q == 0) *(f32x4 *)(out.row_of(s, col) + D) = (f32x4){0, 0, 0, 0};
    }
}

template <int DT, int D, int TILE, int STEP>
static hipError_t launch_reduce(const Kv4AttnArgs &g, hipStream_t st) {
    const unsigned tiles = (unsigned)((int64_t)g.B * g.Hkv * g.col_tiles);
    constexpr int ROWS = 1024 / D;
    if (g.splits <= kFew)
        hipLaunchKernelGGL((kv4_reduce_few_kernel<DT, D, TILE, STEP>),
                           dim3(tiles, (unsigned)((g.part_cols + ROWS - 1) / ROWS)), dim3(256), 0, st, g);
    else
        hipLaunchKernelGGL((kv4_reduce_kernel<DT, D, TILE, STEP>), dim3(tiles, (unsigned)g.part_cols), dim3(256), 0, st,
                           g);
    return hipGetLastError();
}

template <int DT, int D>
static hipError_t launch_reduce_kind(const Kv4AttnArgs &g, hipStream_t st) {
    switch (g.kind) {
        case 0: return launch_reduce<DT, D, 4, 64>(g, st);
        case 1: return launch_reduce<DT, D, 16, 32>(g, st);
        default: return launch_reduce<DT, D, 256, 128>(g, st);
    }
}

hipError_t launch_kv4_reduce(const Kv4AttnArgs &g, hipStream_t st) {
    if (g.D == 128)
        return g.dtype == DT_BF16 ? launch_reduce_kind<DT_BF16, 128>(g, st) : launch_reduce_kind<DT_F16, 128>(g, st);
    return g.dtype == DT_BF16 ? launch_reduce_kind<DT_BF16, 64>(g, st) : launch_reduce_kind<DT_F16, 64>(g, st);
}

}  // namespace awq4
