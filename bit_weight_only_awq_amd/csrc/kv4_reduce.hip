// kv4_reduce.hip -- the sums of an attention call's workgroups, where many share
// a sequence: a kernel after the attention kernel (any of its four forms)
// adds them, writes the rows and clears the workspace.
//
// Bound: latency, and the volume of the partial sums (4 (D + 4) bytes a row
// and workgroup).  One workgroup takes one row, its D/4 quads side by side and
// the splits over the remaining factor of the 256 threads, every load in
// flight at once; the sums are joined in LDS in the splits' order.
#include "kv4_ops.hpp"

namespace awq4 {

template <int DT, int D, int TILE, int STEP>
__global__ __launch_bounds__(256) void kv4_reduce_kernel(Kv4AttnArgs g) {
    constexpr int Q = D / 4, GROUPS = 256 / Q, SHARE = (kKv4MaxSplits + GROUPS - 1) / GROUPS;
    __shared__ f32x4 lds_v[GROUPS][Q];
    __shared__ float lds_r[GROUPS], lds_l[GROUPS];
    const int tile = blockIdx.x, col = blockIdx.y, q = threadIdx.x % Q, group = threadIdx.x / Q;
    const int G = g.Hq / g.Hkv;
    // the attention kernels' order of tiles
    const int bhs = g.B * g.Hkv;
    const int ct = TILE == 256 ? tile / bhs : tile % g.col_tiles, bh = TILE == 256 ? tile % bhs : tile / g.col_tiles;
    const int h = bh % g.Hkv, b = bh / g.Hkv;
    const Kv4Span<TILE, STEP> span(g, b, ct, G);
    if (col >= span.ncols || span.splits == 1) return;
    const AttnRows<DT, D> out{g, tile, span.splits, 0, span.c0, span.q0, h, G};
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
        out.put(col, 4 * q, AttnRows<DT, D>::quotient(v, ll));
    }
    for (int s = group; s < span.splits; s += GROUPS) {
        *(f32x4 *)(out.row_of(s, col) + 4 * q) = (f32x4){0, 0, 0, 0};
        if (q == 0) *(f32x4 *)(out.row_of(s, col) + D) = (f32x4){0, 0, 0, 0};
    }
}

template <int DT, int D, int TILE, int STEP>
static hipError_t launch_reduce(const Kv4AttnArgs &g, hipStream_t st) {
    hipLaunchKernelGGL((kv4_reduce_kernel<DT, D, TILE, STEP>),
                       dim3((unsigned)((int64_t)g.B * g.Hkv * g.col_tiles), (unsigned)g.part_cols), dim3(256), 0, st, g);
    return hipGetLastError();
}

template <int DT, int D>
static hipError_t launch_reduce_kind(const Kv4AttnArgs &g, hipStream_t st) {
    switch (g.kind) {
        case 0: return launch_reduce<DT, D, 4, 64>(g, st);
        case 1: return launch_reduce<DT, D, 16, 32>(g, st);
        case 2: return launch_reduce<DT, D, 32, 32>(g, st);
        default: return launch_reduce<DT, D, 256, 128>(g, st);
    }
}

hipError_t launch_kv4_reduce(const Kv4AttnArgs &g, hipStream_t st) {
    if (g.D == 128)
        return g.dtype == DT_BF16 ? launch_reduce_kind<DT_BF16, 128>(g, st) : launch_reduce_kind<DT_F16, 128>(g, st);
    return g.dtype == DT_BF16 ? launch_reduce_kind<DT_BF16, 64>(g, st) : launch_reduce_kind<DT_F16, 64>(g, st);
}

}  // namespace awq4
