// kv4_decode.hip -- attention over the paged 4-bit cache for at most four query
// rows per key/value head: the answer's next token with groups of up to four
// heads.  Mathematics, masks, splits and reference R as in kv4_attention.hip.
//
// Sixteen columns of a 16 x 16 tile would be twelve or more empty ones, and
// with them most of the exponentials and the arithmetic beside the matrix
// cores, which then bound the kernel (4.3 of the 5.9 TB/s that reading reaches
// here, whatever the number of waves).  So the columns hold four runs of 16
// tokens for four rows: column 4 s + j is row j against the tokens of run s.
// A product's sum over k runs over the four lane groups; the key operand gives
// group g the tokens of run g (eight of their dimensions a product, sixteen
// products for D = 128, as many as before), and the query operand is zero in
// column (s, j) for every group but g = s: each column sums over its own run.
// 64 tokens x 4 rows make one score register quad instead of four.
//
// Loads stay whole lines (a lane reads a quarter of the words of one token in
// each run); a 4 x 4 transpose between lane groups and runs (sixteen lane
// swaps for 64 tokens) puts the tokens of run g into group g.  The scales lie
// where the scores do; the values' zero points move from there to their
// operand by a broadcast along the 16 lanes of a group.  The second product
// takes 32 tokens at a time, two runs, with the probabilities of the other
// columns cleared; its columns stay apart by run until the end, where the
// sixteen partial rows (four waves, four runs) of each row are joined.
//
// Measured (32 heads over 8, D = 128): 64 sequences of 4096 to 8192 tokens 81 us,
// 5.2 TB/s; two of 131072 49 us (and 5 us to add the sums), 5.9 TB/s; 16 of 2050
// with 32 heads of their own 26 us; one of 137 tokens 6.9 us.
#include "kv4_ops.hpp"

namespace awq4 {

// What one wave reads for 64 tokens.
template <int D>
struct Kv4Quad {
    static constexpr int KW = D / 32;
    typedef uint32_t Words __attribute__((ext_vector_type(KW)));
    Words k[4];    // run i: token 16 i + lane % 16, words KW (lane / 16) ..
    u32x4 v[4];    // run i: tokens 4 (lane / 16) .., one word column
    u32x4 km, vm;  // run (lane % 16) / 4: tokens 4 (lane / 16) ..
};

// Registers a and b between the halves (32 lanes) or odd and even rows (16
// lanes) of the wave: a keeps its lower (even) part and takes b's there, b
// takes a's upper (odd) part.
__device__ __forceinline__ void swap32(uint32_t &a, uint32_t &b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = (uint32_t)r[0];
    b = (uint32_t)r[1];
}
__device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = (uint32_t)r[0];
    b = (uint32_t)r[1];
}
// Lane 4 N of each row of 16 lanes, in all of them.
template <int N>
__device__ __forceinline__ uint32_t row_broadcast(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x150 + 4 * N, 0xF, 0xF, false);
}

template <int DT, int D>
__global__ __launch_bounds__(64 * kAttnWaves, 3) void kv4_decode_kernel(Kv4AttnArgs g) {
    using L = Kv4Layout<D>;
    using Quad = Kv4Quad<D>;
    constexpr int KW = D / 32, VM = D / 16, ROW = AttnRows<DT, D>::kRow;
    __shared__ float lds_o[kAttnWaves][16][ROW];
    __shared__ __attribute__((aligned(16))) uint32_t lds_q[5][D / 2 + 4];  // (rows four banks apart)
    __shared__ float lds_row[4][2];  // sum of q, factor of the scores

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, grp = lane >> 4, run = r16 >> 2, j = r16 & 3;
    // workgroup -> (sequence, head), split
    const int tile = blockIdx.x, split = blockIdx.y;
    const int h = tile % g.Hkv, b = tile / g.Hkv;
    const int G = g.Hq / g.Hkv;

    const Kv4Span<4, 64> span(g, b, 0, G);
    const int q0 = span.q0, kv_len = span.kv_len, ncols = span.ncols, splits = span.splits;
    if (ncols <= 0 || split >= splits) return;
    const int s_begin = span.first(split), s_end = span.first(split + 1);
    const int kv_lo = span.kv_lo, kv_hi = span.kv_hi;
    // tokens that all rows see: [all_lo, all_hi)
    const int all_hi = span.pos_of(0, G) + 1;
    const int all_lo = g.window > 0 ? max(span.pos_of(ncols - 1, G) - g.window + 1, 0) : 0;

    const int lgP = __builtin_ctz(g.P);
    const auto *table = (const __attribute__((address_space(4))) int32_t *)(g.tables + (size_t)b * g.table_stride);
    const uint32_t num_pages = (uint32_t)min(g.num_pages, (int64_t)0x7FFFFFFF);
    const uint32_t head_bytes = L::head_words(g.P) * 4, page_bytes = (uint32_t)g.Hkv * head_bytes;
    const char *head = (const char *)g.cache + (size_t)h * head_bytes;
    // this lane's place in a run, in bytes after the run's first word
    const uint32_t k_at = 4 * L::k_word(r16, KW * grp);
    const uint32_t v_at = 4 * L::v_word(g.P, 4 * grp, D == 128 ? r16 : (r16 & 7));
    const uint32_t km_at = 4 * L::k_meta(g.P, 4 * grp), vm_at = 4 * g.P;
    const int last = max(kv_len - 1, 0) >> lgP;
    // the table's entries of the four runs of a step
    struct Entries {
        uint32_t e[4];
    };
    auto entries = [&](int t0) {
        Entries r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.e[i] = (uint32_t)table[min((t0 + 16 * i) >> lgP, last)];
        return r;
    };
    auto load = [&](Quad &s, const Entries &e, int t0) {
        uint32_t mine = 0;  // the page of this lane's scales
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t p = e.e[i] < num_pages ? e.e[i] : 0u, t = (uint32_t)(t0 + 16 * i) & (uint32_t)(g.P - 1);
            const auto page = buf_rsrc(head + (uint64_t)p * page_bytes, head_bytes);
            s.k[i] = buf_get<typename Quad::Words>(page, k_at, t * (4 * L::kWords));
            s.v[i] = buf_get<u32x4>(page, v_at, t * (4 * L::kWords));
            mine = run == i ? p : mine;
        }
        const char *metas = head + (uint64_t)mine * page_bytes + (km_at + 4 * ((uint32_t)(t0 + 16 * run) & (g.P - 1)));
        s.km = *(const u32x4 *)metas;
        s.vm = *(const u32x4 *)(metas + vm_at);
    };

    Quad cur, nxt;
    int st = s_begin + wave;
    Entries now_e{}, next_e{};
    if (st < s_end) {
        now_e = entries(64 * st);
        next_e = entries(64 * (st + kAttnWaves));
        load(cur, now_e, 64 * st);
    }

    // The rows of q, in fp16 and in the order of the operands, in LDS: wave w
    // takes row w, a lane two dimensions (D = 64: the upper lanes none).  A lane
    // reads its column's row in the lane group of its run, and zeros elsewhere.
    if (tid < D / 2) lds_q[4][tid] = 0u;
    {
        const int row = wave < ncols ? wave : 0, qi = row / G, hg = row - qi * G;
        const bool holds = 2 * lane < D;
        const uint32_t *src = (const uint32_t *)((const uint16_t *)g.q + ((size_t)(q0 + qi) * g.Hq + h * G + hg) * D);
        const uint32_t w = holds ? src[lane] : 0u;
        float f[2] = {act_bits_to_f32<DT>(w & 0xFFFFu), act_bits_to_f32<DT>(w >> 16)};
        float mx = fmaxf(fabsf(f[0]), fabsf(f[1]));
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off, 64));
        const int up = query_shift(mx);
        f[0] = __builtin_ldexpf(f[0], up);
        f[1] = __builtin_ldexpf(f[1], up);
        float sum = f[0] + f[1];
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
        const float down = lane & 1 ? 0.0625f : 1.0f;  // columns 2, 3, 6, 7 of a word meet codes times 16
        if (holds) lds_q[wave][lane] = pack_f16(f[0] * down, f[1] * down);
        if (lane == 0) {
            lds_row[wave][0] = sum * 0x1p-24f;
            lds_row[wave][1] = __builtin_ldexpf(g.scale * 1.4426950408889634f, 24 - up);
        }
    }
    __syncthreads();
    const u32x4 *q_from = (const u32x4 *)lds_q[grp == run ? j : 4];
    const float qz = lds_row[j][0], cf = lds_row[j][1];
    const int pos = span.pos_of(j < ncols ? j : 0, G);
    const int hi = pos + 1, lo = g.window > 0 ? pos - g.window + 1 : 0;
    uint32_t mine[4];  // all ones where this lane's column is of run i
#pragma unroll
    for (int i = 0; i < 4; ++i) mine[i] = run == i ? 0xFFFFFFFFu : 0u;

    f32x4 o[VM];
    // (odd waves sum negated probabilities: see kv4_attention.hip)
    const uint32_t odd = wave & 1 ? 0x80008000u : 0u;
    float ref = kNoRef, l = 0.0f;
#pragma unroll
    for (int t = 0; t < VM; ++t) o[t] = (f32x4){0, 0, 0, 0};

    // One step.  there: bit i, run i starts before the end and has a page;
    // plain: all four do, and every row sees every token.
    auto compute = [&](Quad &s, uint32_t there, bool plain, int t0) {
        const int at = t0 + 16 * run + 4 * grp;  // this lane's four tokens
        if (!plain) {
            // tokens that no row sees, or without a page: whatever their meta
            // words hold must not reach the sums
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool any = ((there >> run) & 1) && at + r >= kv_lo && at + r < kv_hi;
                s.km[r] = any ? s.km[r] : 0u;
                s.vm[r] = any ? s.vm[r] : 0u;
            }
        }
        // tokens of run g into lane group g: register i of a word from run i to quarter i
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            uint32_t a = s.k[0][w], b = s.k[1][w], c = s.k[2][w], d = s.k[3][w];
            swap32(a, c);
            swap32(b, d);
            swap16(a, b);
            swap16(c, d);
            s.k[0][w] = a;
            s.k[1][w] = b;
            s.k[2][w] = c;
            s.k[3][w] = d;
        }
        f32x4 x = {0, 0, 0, 0}, x1 = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int w = 0; w < KW; w += 2) {
                x = mfma_f16(word_operand(s.k[i][w]), q_from[KW * i + w], x);
                x1 = mfma_f16(word_operand(s.k[i][w + 1]), q_from[KW * i + w + 1], x1);
            }
        x += x1;
        __builtin_amdgcn_sched_barrier(0);
        float vs[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float ks = act_bits_to_f32<DT>(s.km[r] & 0xFFFFu);
            const float kz = (float)((s.km[r] >> 16) & 0xFFu);
            vs[r] = act_bits_to_f32<DT>(s.vm[r] & 0xFFFFu);
            x[r] = __builtin_fmaf(-kz, qz, x[r]) * ks;
        }
        auto seen = [&](int r) { return ((there >> run) & 1) && at + r >= lo && at + r < hi; };
        float p[4], w[4], top, sum;
        auto numerators = [&] {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                p[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[r], cf, -ref));
                w[r] = p[r] * vs[r];
            }
            if (!plain) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool on = seen(r);
                    p[r] = on ? p[r] : 0.0f;
                    w[r] = on ? w[r] : 0.0f;
                }
            }
            sum = (p[0] + p[1]) + (p[2] + p[3]);
            top = fmaxf(fmaxf(fabsf(w[0]), fabsf(w[1])), fmaxf(fabsf(w[2]), fabsf(w[3])));
        };
        numerators();
        if (__builtin_amdgcn_ballot_w64(!(top <= kMaxP && sum <= kMaxSum)) != 0) {
            float t = -__builtin_inff();
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float y = x[r] * cf;
                const float c = fmaxf(y + __builtin_amdgcn_logf(fabsf(vs[r])) - 11.0f, y - 90.0f);
                t = plain || seen(r) ? fmaxf(t, c) : t;
            }
            t = raised(ref, column_max(t));
            const float f = __builtin_amdgcn_exp2f(ref - t);
            ref = t;
            l *= f;
#pragma unroll
            for (int u = 0; u < VM; ++u) o[u] *= f;
            numerators();
        }
        l += sum;
        const uint32_t p01 = pack_f16(w[0], w[1]) ^ odd, p23 = pack_f16(w[2], w[3]) ^ odd;
        const uint32_t z01 = perm_b32(s.vm[1], s.vm[0], 0x07060302u), z23 = perm_b32(s.vm[3], s.vm[2], 0x07060302u);
        __builtin_amdgcn_sched_barrier(0);
        // runs 0 and 1, then 2 and 3
        static_for<2>([&](auto pair) {
            constexpr int P = 2 * decltype(pair)::value;
            const u32x4 bop = {p01 & mine[P], p23 & mine[P], p01 & mine[P + 1], p23 & mine[P + 1]};
            // the zero points as an operand with equal rows, negative, for
            // operands without and with the factor 16
            const u32x4 z = {row_broadcast<P>(z01), row_broadcast<P>(z23), row_broadcast<P + 1>(z01),
                             row_broadcast<P + 1>(z23)};
            u32x4 z1, z16;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                z1[i] = z[i] | 0x80008000u;
                z16[i] = (z[i] << 4) | 0x80008000u;
            }
            const ValuePairs<D> pairs(s.v[P], s.v[P + 1], r16);
#pragma unroll
            for (int t = 0; t < VM; ++t) {
                o[t] = mfma_f16(pairs.operand(t), bop, mfma_f16(value_pos<D>(t) & 1 ? z16 : z1, bop, o[t]));
                if (t & 1) __builtin_amdgcn_sched_barrier(0);
            }
        });
    };

    auto step = [&](Quad &now, Quad &next) {
        const int t0 = 64 * st;
        uint32_t there = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) there |= (uint32_t)(now_e.e[i] < num_pages && t0 + 16 * i < kv_len) << i;
        const bool plain = there == 15 && t0 >= all_lo && t0 + 64 <= all_hi;
        st += kAttnWaves;
        now_e = next_e;
        if (st < s_end) {
            load(next, now_e, 64 * st);
            next_e = entries(64 * (st + kAttnWaves));
        }
        compute(now, there, plain, t0);
    };
    while (st < s_end) {
        step(cur, nxt);
        if (st >= s_end) break;
        step(nxt, cur);
    }

    const AttnRows<DT, D> out{g, tile, splits, split, 0, q0, h, G};
    const float lsum = column_sum(l);
    float *part = &lds_o[wave][r16][0];
#pragma unroll
    for (int t = 0; t < VM; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) part[value_dim<D>(t, 4 * grp + r)] = o[t][r] * (odd ? -value_unit<D>(t) : value_unit<D>(t));
    if (grp == 0) {
        part[D] = ref;
        part[D + 1] = lsum;
    }
    __syncthreads();
    // (partial 4 w + s of row j: wave w, column 4 s + j)
    out.template join<4 * kAttnWaves>(&lds_o[0][0][0], [](int p, int col) { return 4 * p + col; }, 0, ncols);
}

template <int DT, int D>
static hipError_t launch_decode(const Kv4AttnArgs &g, hipStream_t st) {
    hipLaunchKernelGGL((kv4_decode_kernel<DT, D>), dim3((unsigned)((int64_t)g.B * g.Hkv), (unsigned)g.splits),
                       dim3(64 * kAttnWaves), 0, st, g);
    return hipGetLastError();
}

hipError_t launch_kv4_decode(const Kv4AttnArgs &g, hipStream_t st) {
    if (g.D == 128)
        return g.dtype == DT_BF16 ? launch_decode<DT_BF16, 128>(g, st) : launch_decode<DT_F16, 128>(g, st);
    return g.dtype == DT_BF16 ? launch_decode<DT_BF16, 64>(g, st) : launch_decode<DT_F16, 64>(g, st);
}

}  // namespace awq4
