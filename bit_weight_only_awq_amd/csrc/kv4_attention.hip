// kv4_attention.hip -- causal attention over the paged 4-bit cache (layout:
// kv4.hpp) for few query rows per key/value head: decode, several tokens at
// once, short chunks.
//
// Query i of a sequence with n new tokens and L tokens in all stands at
// position p = L - n + i and sees the keys j <= p (with a window w: j > p - w).
//   t_j = scale s_j (Q . c_j - z_j sum_d Q_d)
//   O   = sum_j softmax(t)_j s'_j (c'_j - z'_j)
// with codes c, zero points z and scales s of the keys, primed ones of the
// values.  The codes enter the matrix cores as they are: a masked pair of
// nibbles is a pair of fp16 subnormals, exactly c 2^-24 (16 c 2^-24 for the
// upper nibble of a byte), one AND and no conversion.  Scales and zero points
// act on the fp32 scores, and on the value side the scale is folded into the
// probabilities, whose one rounding (to fp16, the matrix cores' type; the
// values' codes are exact in it) is the only one between q and the output's:
//   p_j = 2^(t_j log2(e) - R),  P_j = fp16(p_j s'_j)
//   O = (sum P_j c'_j - sum P_j z'_j) / sum p_j
// The reference R of a row is raised when a |P_j| would pass 2^15 (or a p_j 2^100,
// for values whose scale is next to nothing), to put the largest at 2^11: P
// then uses fp16's whole range, and one 2^-25 times the largest still has all 11
// bits, whatever the scales' magnitude.  Most steps find nothing to raise and
// need no exchange between lanes.  The sum of z' takes the rounded P, so that
// a code and its zero point lose the same, and it is taken off step by step:
// codes average 7.5, and of the sums of long contexts little is left after 7.5
// has gone.  For the same reason it shows that the matrix cores drop the bits
// of a product far below the largest of its sum, always downwards: every other
// wave sums negated probabilities, whose loss is upwards.  (Error of the output
// for 131072 tokens, its own rounding to 11 bits 2.0e-4: zero points taken off
// at the end 8.4e-4, step by step 5.5e-4, with half the waves negated 2.7e-4.)
// Queries are scaled by a power of two to just below 2^15 before they become
// fp16: exact for fp16 and for bf16 (8 bits), down to 2^-25 of a row's largest
// (bf16 rows that are below 2^-86 throughout keep fewer bits).
//
// Tiles are transposed, S^T = K Q^T and O^T = V^T P^T: the lanes of a column
// (one query row) hold the scores of the tokens that they then need as the
// second product's operand, so probabilities never move between lanes.  16
// tokens x 16 query rows a tile; the rows of a sequence and key/value head are
// its (new token, head of the group) pairs.
//
// Bound: device memory (D + 8 bytes a token and head, read once).  A workgroup
// of four waves takes a run of tokens, each wave 32 of every 128; the four
// join their sums through LDS, and the workgroups of a sequence (as many as
// its length asks for, known only on the device) leave theirs in the workspace
// for kv4_reduce.hip.  Measured (32 heads over 8, D = 128, bf16): 16 sequences of
// 4096 tokens, 8 rows a head 21 us, 16 rows 22, 64 rows 51, 128 rows (two tiles
// of 16 a workgroup) 66; one of 8192, 64 rows 18.  (Eight rows take nearly the
// time of sixteen: their tile's other columns are computed too.)
#include "kv4_ops.hpp"

namespace awq4 {

// What one wave reads for 32 tokens: two tiles of 16.
template <int D>
struct Kv4Step {
    static constexpr int KW = D / 32;  // words of a token in a lane
    typedef uint32_t Words __attribute__((ext_vector_type(KW)));
    Words k[2];
    u32x4 v[2], km[2], vm[2];
};

template <int DT, int D, int NT>
__global__ __launch_bounds__(64 * kAttnWaves, NT == 1 ? 3 : 2) void kv4_attention_kernel(Kv4AttnArgs g) {
    using L = Kv4Layout<D>;
    using Step = Kv4Step<D>;
    constexpr int COLS = 16 * NT, KW = D / 32, VM = D / 16, ROW = AttnRows<DT, D>::kRow;
    __shared__ float lds_o[kAttnWaves][16][ROW];  // one 16-column tile of every wave; at D its R, at D + 1 its sum of p

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, grp = lane >> 4;
    // workgroup -> (sequence, head, column tile), split
    const int tile = blockIdx.x, split = blockIdx.y;
    const int ct = tile % g.col_tiles, bh = tile / g.col_tiles;
    const int h = bh % g.Hkv, b = bh / g.Hkv;
    const int G = g.Hq / g.Hkv;

    const Kv4Span<COLS, 32> span(g, b, ct, G);
    const int q0 = span.q0, kv_len = span.kv_len, c0 = span.c0, ncols = span.ncols;
    const int splits = NT == 2 ? 1 : span.splits;  // (tiles of 32 rows are taken where they fill the device unsplit)
    if (ncols <= 0 || split >= splits) return;
    const int s_begin = span.first(split), s_end = span.first(split + 1);
    const int kv_lo = span.kv_lo, kv_hi = span.kv_hi;
    // tokens that all of the tile's rows see: [all_lo, all_hi)
    const int all_hi = span.pos_of(c0, G) + 1;
    const int all_lo = g.window > 0 ? max(span.pos_of(c0 + ncols - 1, G) - g.window + 1, 0) : 0;

    const int lgP = __builtin_ctz(g.P);
    // (in the constant address space: no kernel of this call writes it, so it is
    // read through the scalar cache)
    const auto *table = (const __attribute__((address_space(4))) int32_t *)(g.tables + (size_t)b * g.table_stride);
    const uint32_t num_pages = (uint32_t)min(g.num_pages, (int64_t)0x7FFFFFFF);
    const uint32_t page_bytes = (uint32_t)g.Hkv * L::head_words(g.P) * 4;
    const uint32_t head_bytes = L::head_words(g.P) * 4;
    const char *head = (const char *)g.cache + (size_t)h * head_bytes;
    // this lane's place in a tile of 16 tokens, in bytes after the tile's first word
    const uint32_t k_at = 4 * L::k_word(r16, KW * grp), m_at = 16 * grp;
    const uint32_t v_at = 4 * L::v_word(g.P, 4 * grp, D == 128 ? r16 : (r16 & 7));
    const uint32_t km_at = 4 * L::k_meta(g.P, 0) + m_at, vm_at = 4 * L::v_meta(g.P, 0) + m_at;
    // the table's entries for the two tiles of a step (past the end: the last
    // token's), and whether a tile's first token is there and has a page
    const int last = max(kv_len - 1, 0) >> lgP;
    auto entry = [&](int t) { return (uint32_t)table[min(t >> lgP, last)]; };
    auto there = [&](uint32_t e, int t) { return e < num_pages && t < kv_len; };
    auto load = [&](Step &s, uint32_t e0, uint32_t e1, int t0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t e = i ? e1 : e0, t = (uint32_t)(t0 + 16 * i) & (uint32_t)(g.P - 1);
            // (a buffer descriptor a tile: scalar base and offset plus a 32-bit
            // lane offset, no 64-bit sums per lane)
            const auto page = buf_rsrc(head + (uint64_t)(e < num_pages ? e : 0u) * page_bytes, head_bytes);
            s.k[i] = buf_get<typename Step::Words>(page, k_at, t * (4 * L::kWords));
            s.v[i] = buf_get<u32x4>(page, v_at, t * (4 * L::kWords));
            s.km[i] = buf_get<u32x4>(page, km_at, 4 * t);
            s.vm[i] = buf_get<u32x4>(page, vm_at, 4 * t);
        }
    };

    // the first step's loads before anything else
    Step cur, nxt;
    int st = s_begin + wave;
    uint32_t e0 = 0, e1 = 0, n0 = 0, n1 = 0;  // this step's entries, the next one's
    if (st < s_end) {
        e0 = entry(32 * st);
        e1 = entry(32 * st + 16);
        n0 = entry(32 * (st + kAttnWaves));
        n1 = entry(32 * (st + kAttnWaves) + 16);
        load(cur, e0, e1, 32 * st);
    }

    // this lane's columns: their rows of q as matrix-core operand, in fp16
    u32x4 qf[NT][KW];
    float qz[NT], cf[NT];
    int lo[NT], hi[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int col = 16 * n + r16;
        const bool live = col < ncols;
        const int row = c0 + (live ? col : 0);
        const int qi = row / G, hg = row - qi * G;
        const int pos = span.pos_of(row, G);
        hi[n] = pos + 1;
        lo[n] = g.window > 0 ? pos - g.window + 1 : 0;
        const uint16_t *src = (const uint16_t *)g.q + ((size_t)(q0 + qi) * g.Hq + h * G + hg) * D + 8 * KW * grp;
        float f[KW][8], mx = 0.0f;
#pragma unroll
        for (int i = 0; i < KW; ++i) {
            const u32x4 w = *(const u32x4 *)(src + 8 * i);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[i][e] = live ? act_bits_to_f32<DT>((w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu) : 0.0f;
                mx = fmaxf(mx, fabsf(f[i][e]));
            }
        }
        mx = column_max(mx);
        const int up = query_shift(mx);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < KW; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[i][e] = __builtin_ldexpf(f[i][e], up);
                sum += f[i][e];
            }
            qf[n][i] = query_operand(f[i]);
        }
        qz[n] = column_sum(sum) * 0x1p-24f;
        cf[n] = __builtin_ldexpf(g.scale * 1.4426950408889634f, 24 - up);
    }

    f32x4 o[NT][VM];
    // (odd waves sum negated probabilities: see above)
    const uint32_t odd = wave & 1 ? 0x80008000u : 0u;
    float ref[NT], l[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        ref[n] = kNoRef;
        l[n] = 0.0f;
#pragma unroll
        for (int t = 0; t < VM; ++t) o[n][t] = (f32x4){0, 0, 0, 0};
    }
    // One step.  plain: every token of it is there and every column sees it.
    auto compute = [&](Step &s, bool plain, bool in0, bool in1, int t0) {
        if (!plain) {
            // tokens that no column sees, or without a page: whatever their
            // meta words hold must not reach the sums
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = t0 + 16 * i + 4 * grp + r;
                    const bool any = (i ? in1 : in0) && j >= kv_lo && j < kv_hi;
                    s.km[i][r] = any ? s.km[i][r] : 0u;
                    s.vm[i][r] = any ? s.vm[i][r] : 0u;
                }
        }
        f32x4 x[NT][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int n = 0; n < NT; ++n) x[n][i] = (f32x4){0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < KW; ++j) {
                const u32x4 a = word_operand(s.k[i][j]);
#pragma unroll
                for (int n = 0; n < NT; ++n) x[n][i] = mfma_f16(a, qf[n][j], x[n][i]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        float vs[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float ks = act_bits_to_f32<DT>(s.km[i][r] & 0xFFFFu);
                const float kz = (float)((s.km[i][r] >> 16) & 0xFFu);
                vs[i][r] = act_bits_to_f32<DT>(s.vm[i][r] & 0xFFFFu);
#pragma unroll
                for (int n = 0; n < NT; ++n) x[n][i][r] = __builtin_fmaf(-kz, qz[n], x[n][i][r]) * ks;
            }
        u32x4 pf[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            auto seen = [&](int i, int r) {
                const int j = t0 + 16 * i + 4 * grp + r;
                return (i ? in1 : in0) && j >= lo[n] && j < hi[n];
            };
            float p[2][4], w[2][4], top, sum;
            auto numerators = [&] {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        p[i][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[n][i][r], cf[n], -ref[n]));
                        w[i][r] = p[i][r] * vs[i][r];
                    }
                if (!plain) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const bool on = seen(i, r);
                            p[i][r] = on ? p[i][r] : 0.0f;
                            w[i][r] = on ? w[i][r] : 0.0f;
                        }
                }
                top = sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        sum += p[i][r];
                        top = fmaxf(top, fabsf(w[i][r]));
                    }
            };
            numerators();
            if (__builtin_amdgcn_ballot_w64(!(top <= kMaxP && sum <= kMaxSum)) != 0) {
                float t = -__builtin_inff();
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float y = x[n][i][r] * cf[n];
                        const float c = fmaxf(y + __builtin_amdgcn_logf(fabsf(vs[i][r])) - 11.0f, y - 90.0f);
                        t = plain || seen(i, r) ? fmaxf(t, c) : t;
                    }
                t = raised(ref[n], column_max(t));
                const float f = __builtin_amdgcn_exp2f(ref[n] - t);
                ref[n] = t;
                l[n] *= f;
#pragma unroll
                for (int u = 0; u < VM; ++u) o[n][u] *= f;
                numerators();
            }
            l[n] += sum;
            pf[n] = (u32x4){pack_f16(w[0][0], w[0][1]) ^ odd, pack_f16(w[0][2], w[0][3]) ^ odd,
                            pack_f16(w[1][0], w[1][1]) ^ odd, pack_f16(w[1][2], w[1][3]) ^ odd};
        }
        __builtin_amdgcn_sched_barrier(0);
        // the values' zero points as an operand with equal rows, negative, for
        // columns without and with the factor 16
        u32x4 z1, z16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t z =
                perm_b32(s.vm[i >> 1][2 * (i & 1) + 1], s.vm[i >> 1][2 * (i & 1)], 0x07060302u);
            z1[i] = z | 0x80008000u;
            z16[i] = (z << 4) | 0x80008000u;
        }
        const ValuePairs<D> pairs(s.v[0], s.v[1], r16);
#pragma unroll
        for (int t = 0; t < VM; ++t) {
            const u32x4 a = pairs.operand(t);
#pragma unroll
            for (int n = 0; n < NT; ++n)
                o[n][t] = mfma_f16(a, pf[n], mfma_f16(value_pos<D>(t) & 1 ? z16 : z1, pf[n], o[n][t]));
            if (t & 1) __builtin_amdgcn_sched_barrier(0);
        }
    };

    // Two steps in turn, each with registers of its own: the loads of one are
    // in flight while the other is computed (a copy from one to the other would
    // wait for them).
    auto run = [&](Step &now, Step &next) {
        const int t0 = 32 * st;
        const bool in0 = there(e0, t0), in1 = there(e1, t0 + 16);
        const bool plain = in0 && in1 && t0 >= all_lo && t0 + 32 <= all_hi;
        st += kAttnWaves;
        e0 = n0;
        e1 = n1;
        if (st < s_end) {
            load(next, e0, e1, 32 * st);
            n0 = entry(32 * (st + kAttnWaves));
            n1 = entry(32 * (st + kAttnWaves) + 16);
        }
        compute(now, plain, in0, in1, t0);
    };
    while (st < s_end) {
        run(cur, nxt);
        if (st >= s_end) break;
        run(nxt, cur);
    }

    // Join the four waves, 16 columns at a time.
    const AttnRows<DT, D> out{g, tile, splits, split, c0, q0, h, G};
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int nc = min(16, ncols - 16 * n);
        if (nc <= 0) break;
        if (n) __syncthreads();
        const float lsum = column_sum(l[n]);
        float *mine = &lds_o[wave][r16][0];
#pragma unroll
        for (int t = 0; t < VM; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) mine[value_dim<D>(t, 4 * grp + r)] = o[n][t][r] * (odd ? -value_unit<D>(t) : value_unit<D>(t));
        if (grp == 0) {
            mine[D] = ref[n];
            mine[D + 1] = lsum;
        }
        __syncthreads();
        out.template join<kAttnWaves>(&lds_o[0][0][0], [](int w, int col) { return 16 * w + col; }, 16 * n, nc);
    }
}

template <int DT, int D, int NT>
static hipError_t launch_attn(const Kv4AttnArgs &g, hipStream_t st) {
    hipLaunchKernelGGL((kv4_attention_kernel<DT, D, NT>),
                       dim3((unsigned)((int64_t)g.B * g.Hkv * g.col_tiles), (unsigned)g.splits), dim3(64 * kAttnWaves),
                       0, st, g);
    return hipGetLastError();
}

template <int DT, int D>
static hipError_t launch_attn_nt(const Kv4AttnArgs &g, hipStream_t st) {
    return g.kind == 1 ? launch_attn<DT, D, 1>(g, st) : launch_attn<DT, D, 2>(g, st);
}

hipError_t launch_kv4_attention(const Kv4AttnArgs &g, hipStream_t st) {
    if (g.D == 128)
        return g.dtype == DT_BF16 ? launch_attn_nt<DT_BF16, 128>(g, st) : launch_attn_nt<DT_F16, 128>(g, st);
    return g.dtype == DT_BF16 ? launch_attn_nt<DT_BF16, 64>(g, st) : launch_attn_nt<DT_F16, 64>(g, st);
}

}  // namespace awq4
