// kv4_prefill.hip -- causal attention over the paged 4-bit cache (layout:
// kv4.hpp, mathematics and masks: kv4_attention.hip) for many query rows per
// key/value head: prompts and chunks of prompts.
//
// Bound: the matrix cores (4 D flops a row and token) and, at the same rate,
// the vector units, which take an exponential and about five more
// instructions a row and token.  So what a token costs is paid once for many
// rows: a workgroup takes 128 rows of a sequence and key/value head (the heads
// of a group side by side, so that they share the unpacking), 32 a wave, and
// 64 tokens at a time go through LDS as 16-bit integers (code - zero point),
// exact in either 16-bit type; each wave unpacks 16 tokens for all four.
// Nothing is left of the zero points then, and a score costs one FMA:
//   p_j = 2^(x_j (scale log2(e) s_j) - R),  x_j = q . (c_j - z_j)
// with q as it came (fp16 or bf16 operands by its type); the second product
// is fp16 for both (probabilities with the values' scales, 11 bits; see
// kv4_attention.hip for R).  Transposed 32 x 32 tiles, S^T = K Q^T and O^T =
// V^T P^T: a lane's scores are its own operand of the second product.  V lies
// in LDS by dimension, the tokens of a row in the order in which S^T's rows
// fall to a lane.  Tiles are double-buffered: the words of a tile are loaded
// two tiles ahead and unpacked one ahead, one barrier a tile.  Two workgroups
// (64 KB each at D = 128) share a CU, out of step, so that one's exponentials
// run beside the other's matrix products.
#include "kv4_ops.hpp"

namespace awq4 {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kPreWaves = 4, kPreTile = 64;  // waves (32 rows each) and tokens of a tile

template <int DT>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    if (DT == DT_F16) return __builtin_amdgcn_mfma_f32_32x32x16_f16(bit_as<f16x8>(a), bit_as<f16x8>(b), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(bit_as<bf16x8>(a), bit_as<bf16x8>(b), c, 0, 0, 0);
}

// Of the two lanes of a column (l, l ^ 32): the larger value, the sum.
__device__ __forceinline__ float pair_max(float v) {
    const auto h = __builtin_amdgcn_permlane32_swap(bit_as<uint32_t>(v), bit_as<uint32_t>(v), false, false);
    return fmaxf(bit_as<float>((uint32_t)h[0]), bit_as<float>((uint32_t)h[1]));
}
__device__ __forceinline__ float pair_sum(float v) {
    const auto h = __builtin_amdgcn_permlane32_swap(bit_as<uint32_t>(v), bit_as<uint32_t>(v), false, false);
    return bit_as<float>((uint32_t)h[0]) + bit_as<float>((uint32_t)h[1]);
}

// One tile in LDS, in bytes: keys [64][D] and values [D][64] as 16-bit
// integers, then the keys' scales times scale log2(e) and the values'.  Rows are 128 or 256 bytes, so their 16-byte chunks
// are permuted by the row's number: the lanes that an access serves at once
// read rows one apart and write rows one or eight apart.  Chunk c of row r is
// at row(r) ^ (c << 4): one instruction from a per-lane base.
template <int D>
struct PreTile {
    static constexpr uint32_t kV = 2 * kPreTile * D, kKs = 2 * kV, kVs = kKs + 4 * kPreTile,
                              kBytes = kVs + 4 * kPreTile + (256 - 8 * kPreTile % 256) % 256;
    __device__ static uint32_t mix(uint32_t r) { return (r ^ (r >> 3)) & 7; }
    __device__ static uint32_t k_row(uint32_t t) { return 2 * D * t + 16 * (D == 128 ? t & 15 : mix(t)); }
    __device__ static uint32_t v_row(uint32_t d) { return kV + 2 * kPreTile * d + 16 * mix(d); }
};
typedef __attribute__((address_space(3))) char *LdsPtr;
template <typename T>
__device__ __forceinline__ T lds_get(uint32_t at) {
    return *(const __attribute__((address_space(3))) T *)(LdsPtr)(uintptr_t)at;
}
template <typename T>
__device__ __forceinline__ void lds_put(uint32_t at, T v) {
    *(__attribute__((address_space(3))) T *)(LdsPtr)(uintptr_t)at = v;
}

// What a thread holds of a tile before it is unpacked: a quarter of one
// token's keys, and one word column of four tokens' values.
template <int D>
struct PreRaw {
    typedef uint32_t Words __attribute__((ext_vector_type(D / 32)));
    Words k;
    u32x4 v, vm;
    uint32_t km, vm1;  // the token's own metas; vm: the four tokens'
};

template <int DT, int D>
__global__ __launch_bounds__(64 * kPreWaves, 2) void kv4_prefill_kernel(Kv4AttnArgs g) {
    using L = Kv4Layout<D>;
    using Raw = PreRaw<D>;
    constexpr int COLS = 32 * kPreWaves, KS = D / 16, DTL = D / 32, ROW = D + 4;
    using Tile = PreTile<D>;
    __shared__ __attribute__((aligned(256))) char lds[2 * Tile::kBytes];
    const uint32_t lds0 = lds_address(lds);

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c32 = lane & 31, half = lane >> 5;
    const int ct = g.col_tiles - 1 - (int)(blockIdx.x / (g.B * g.Hkv)), bh = blockIdx.x % (g.B * g.Hkv);
    const int h = bh % g.Hkv, b = bh / g.Hkv, split = blockIdx.y;
    const int G = g.Hq / g.Hkv;

    const Kv4Span<COLS, kPreTile> span(g, b, ct, G);
    const int q0 = span.q0, kv_len = span.kv_len, c0 = span.c0, ncols = span.ncols, splits = span.splits;
    if (ncols <= 0 || split >= splits) return;
    const int t_begin = span.first(split), t_end = span.first(split + 1);
    const int kv_lo = span.kv_lo, kv_hi = span.kv_hi;
    // tokens that any row of this wave sees, and that all of them see
    const int w0 = c0 + 32 * wave, w1 = min(w0 + 32, c0 + ncols);  // w1 <= w0: no rows
    const int first_pos = span.pos_of(w0, G), last_pos = span.pos_of(max(w1, w0 + 1) - 1, G);
    const int wave_hi = w1 > w0 ? last_pos + 1 : 0, wave_lo = g.window > 0 ? first_pos - g.window + 1 : 0;
    const int all_hi = first_pos + 1, all_lo = g.window > 0 ? last_pos - g.window + 1 : 0;

    // this lane's row
    const int row = min(w0 + c32, c0 + ncols - 1), qi = row / G, hg = row - qi * G;
    const int hi = span.pos_of(row, G) + 1, lo = g.window > 0 ? hi - g.window : 0;
    const size_t row_at = ((size_t)(q0 + qi) * g.Hq + h * G + hg) * D;
    u32x4 qf[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) qf[i] = *(const u32x4 *)((const uint16_t *)g.q + row_at + 16 * i + 8 * half);

    const int lgP = __builtin_ctz(g.P);
    const auto *table = (const __attribute__((address_space(4))) int32_t *)(g.tables + (size_t)b * g.table_stride);
    const int64_t page_bytes = (int64_t)g.Hkv * L::head_words(g.P) * 4;
    const char *head = (const char *)g.cache + (int64_t)h * L::head_words(g.P) * 4;
    auto page_of = [&](int t) -> int {
        if (t >= kv_len) return -1;
        const int p = __builtin_amdgcn_readfirstlane(table[t >> lgP]);
        return p >= 0 && p < g.num_pages ? p : -1;
    };
    // this wave unpacks tokens 16 wave .. of a tile: a lane has token lane / 4
    // and a quarter of its key words, and the value words of tokens 4 vg ..
    // 4 vg + 3 in column vw (D = 64: the upper lanes repeat the lower ones')
    const int kt = lane >> 2, kq = lane & 3;
    const int vw = lane & (L::kWords - 1), vg = (lane / L::kWords) & 3;
    const uint32_t k_at = 4 * L::k_word(kt, (D / 32) * kq), v_at = 4 * L::v_word(g.P, 4 * vg, vw);
    const uint32_t km_at = 4 * L::k_meta(g.P, kt), vm1_at = 4 * L::v_meta(g.P, kt), vm_at = 4 * L::v_meta(g.P, 4 * vg);
    const float score_scale = g.scale * 1.4426950408889634f;

    auto load = [&](Raw &r, int tile) {
        const int t = kPreTile * tile + 16 * wave;
        const int page = page_of(t), in = t & (g.P - 1);
        const char *at = head + max(page, 0) * page_bytes;
        const char *words = at + in * (4 * L::kWords), *metas = at + 4 * in;
        r.k = *(const typename Raw::Words *)(words + k_at);
        r.v = *(const u32x4 *)(words + v_at);
        r.km = *(const uint32_t *)(metas + km_at);
        r.vm1 = *(const uint32_t *)(metas + vm1_at);
        r.vm = *(const u32x4 *)(metas + vm_at);
        // tokens that no row sees, or without a page
        if (page < 0 || t < kv_lo || t + 16 > kv_hi) {
            auto there = [&](int j) { return page >= 0 && j >= kv_lo && j < kv_hi; };
            r.km = there(t + kt) ? r.km : 0u;
            r.vm1 = there(t + kt) ? r.vm1 : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) r.vm[i] = there(t + 4 * vg + i) ? r.vm[i] : 0u;
        }
    };
    // this lane's rows, less the buffer: written (key token, value dimension 8
    // vw, in the chunk of its four tokens) and read (key token, value dimension c32)
    const int vn = 4 * wave + vg;
    const uint32_t k_put = Tile::k_row(16 * wave + kt) ^ (16 * (D / 32) * kq);
    const uint32_t v_put = (Tile::v_row(8 * vw) ^ (16 * (2 * (vn >> 2) + (vn & 1)))) + 8 * ((vn >> 1) & 1);
    const uint32_t k_get = Tile::k_row(c32) ^ (16 * half), v_get = Tile::v_row(c32) ^ (16 * half);
    auto unpack = [&](const Raw &r, uint32_t buf) {
        const int t = 16 * wave + kt;
        // keys: word i of the quarter is chunk (D/32) kq + i of the token's row
        const uint32_t z = (r.km >> 16) & 15u;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint32_t w = r.k[i];
            u32x4 o;
            if (DT == DT_F16) {
                const f16x2 one = {(f16)1.0f, (f16)1.0f}, s16 = {(f16)0.0625f, (f16)0.0625f};
                const f16x2 zl = bit_as<f16x2>(zconst_f16<0>(z)), zh = bit_as<f16x2>(zconst_f16<1>(z));
                const uint32_t u = w >> 8;
                o[0] = bit_as<uint32_t>(bit_as<f16x2>((w & 0x000F000Fu) | 0x64006400u) * one + zl);
                o[1] = bit_as<uint32_t>(bit_as<f16x2>((w & 0x00F000F0u) | 0x64006400u) * s16 + zh);
                o[2] = bit_as<uint32_t>(bit_as<f16x2>((u & 0x000F000Fu) | 0x64006400u) * one + zl);
                o[3] = bit_as<uint32_t>(bit_as<f16x2>((u & 0x00F000F0u) | 0x64006400u) * s16 + zh);
            } else {
                // (integers up to 15 in bf16; bytes 0..3 of e hold nibbles 0, 2, 4, 6, those of o 1, 3, 5, 7)
                typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                const float zf = (float)z;
                const uint32_t e = w & 0x0F0F0F0Fu, d = (w >> 4) & 0x0F0F0F0Fu;
                auto two = [&](uint32_t x, int lo8) {
                    const f32x2 f = {(float)((x >> lo8) & 0xFFu) - zf, (float)((x >> (lo8 + 16)) & 0xFFu) - zf};
                    return bit_as<uint32_t>(__builtin_convertvector(f, bf16x2));
                };
                o = (u32x4){two(e, 0), two(d, 0), two(e, 8), two(d, 8)};
            }
            lds_put(buf + (k_put ^ (16 * i)), o);
        }
        if (kq == 0) {
            // a value scale that is no number moves to the score: rows that do
            // not see the token clear the score's exponential, and 0 * NaN
            // would bring it back
            const float vs = act_bits_to_f32<DT>(r.vm1 & 0xFFFFu);
            lds_put(buf + Tile::kKs + 4 * t, vs == vs ? act_bits_to_f32<DT>(r.km & 0xFFFFu) * score_scale : vs);
        }
        // values: tokens 4 vn .. 4 vn + 3 of the tile are S^T rows of the lanes'
        // half vn & 1, the first or second four by vn & 2, in the 16-token step
        // vn >> 2: that is their chunk of a dimension's row and place in it
        uint32_t zl[2], zh[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t zz = perm_b32(r.vm[2 * i + 1], r.vm[2 * i], 0x07060302u) & 0x000F000Fu;
            zl[i] = 0xE400E400u | zz;         // -(1024 + z)
            zh[i] = 0xD400D400u | (zz << 4);  // -(64 + z)
        }
        if (D == 128 || lane < 32) {
#pragma unroll
            for (int t8 = 0; t8 < 8; ++t8) {
                u32x2 o;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t w = t8 & 1 ? pair_y(r.v[2 * i], r.v[2 * i + 1]) : pair_x(r.v[2 * i], r.v[2 * i + 1]);
                    if (col_shift(t8)) w >>= 8;
                    const f16x2 s16 = {(f16)0.0625f, (f16)0.0625f};
                    if (col_hi(t8))
                        o[i] = bit_as<uint32_t>(bit_as<f16x2>((w & 0x00F000F0u) | 0x64006400u) * s16 +
                                                bit_as<f16x2>(zh[i]));
                    else
                        o[i] = bit_as<uint32_t>(bit_as<f16x2>((w & 0x000F000Fu) | 0x64006400u) + bit_as<f16x2>(zl[i]));
                }
                lds_put(buf + (v_put ^ (16 * t8)) + 2 * kPreTile * t8, o);
            }
            if (vw == 0) {
                f32x4 f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float vs = act_bits_to_f32<DT>(r.vm[i] & 0xFFFFu);
                    f[i] = vs == vs ? vs : 0.0f;
                }
                lds_put(buf + Tile::kVs + 16 * vn, f);
            }
        }
    };

    f32x16 o[DTL];
    float ref = kNoRef, l = 0.0f;
#pragma unroll
    for (int i = 0; i < DTL; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;

    // One tile.  there: its four runs of 16 tokens have a page; plain: all of
    // them, and every row of the wave sees every token.  A raised reference
    // takes the scores' products again rather than keep them beside p.
    auto compute = [&](uint32_t buf, int t0, const bool (&there)[4], bool plain) {
        // (opaque, so that the sixteen addresses made from each are not all kept across tiles)
        uint32_t k_from = buf + k_get, v_from = buf + v_get;
        asm("" : "+v"(k_from), "+v"(v_from));
        const uint32_t s_from = buf + 16 * half;
        // token of register 4 a + r of tile u: 32 u + 8 a + 4 half + r
        const int at = t0 + 4 * half - lo, span = max(hi - lo, 0);
        // (opaque where used, so that the 32 comparisons are not kept from one use to the next)
        auto seen = [&](int u, int a, int r, int from) {
            return (unsigned)(from + 32 * u + 8 * a + r) < (unsigned)span && there[2 * u + a / 2];
        };
        auto opaque = [](int v) {
            asm volatile("" : "+v"(v));
            return v;
        };
        f32x16 x[2];
        uint32_t pf[2][8];
        float sum;
        bool raise = __builtin_amdgcn_ballot_w64(ref == kNoRef) != 0;  // rows that have seen nothing yet
        while (true) {
            const float from_ref = ref == kNoRef ? 0.0f : ref;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int r = 0; r < 16; ++r) x[u][r] = 0.0f;
#pragma unroll
                for (int i = 0; i < KS; ++i)
                    x[u] = mfma32<DT>(lds_get<u32x4>((k_from ^ (32 * i) ^ (D == 64 ? 64 * u : 0)) + 64 * D * u), qf[i],
                                      x[u]);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const f32x4 ks = lds_get<f32x4>(s_from + Tile::kKs + 128 * u + 32 * a);
#pragma unroll
                    for (int r = 0; r < 4; ++r) x[u][4 * a + r] = __builtin_fmaf(x[u][4 * a + r], ks[r], -from_ref);
                }
            __builtin_amdgcn_sched_barrier(0);
            if (raise) {
                float m = ref == kNoRef ? kNoRef : 0.0f;
                const int from = opaque(at);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        const f32x4 vs = lds_get<f32x4>(s_from + Tile::kVs + 128 * u + 32 * a);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float y = x[u][4 * a + r];
                            const float c = fmaxf(y + __builtin_amdgcn_logf(vs[r]) - 11.0f, y - 90.0f);
                            m = plain || seen(u, a, r, from) ? fmaxf(m, c) : m;
                        }
                    }
                m = pair_max(m);
                const float f = m > 0.0f ? __builtin_amdgcn_exp2f(-m) : 1.0f;  // (a first reference: o and l are 0)
                ref = m == kNoRef ? kNoRef : from_ref + m;
                l *= f;
#pragma unroll
                for (int i = 0; i < DTL; ++i) o[i] *= f;
#pragma unroll
                for (int u = 0; u < 2; ++u) x[u] -= m;
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r) x[u][r] = __builtin_amdgcn_exp2f(x[u][r]);
            if (!plain) {
                const int from = opaque(at);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int r = 0; r < 16; ++r) x[u][r] = seen(u, r / 4, r % 4, from) ? x[u][r] : 0.0f;
            }
            float top = 0.0f;
            sum = 0.0f;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const f32x4 vs = lds_get<f32x4>(s_from + Tile::kVs + 128 * u + 32 * a);
                    float w[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        w[r] = x[u][4 * a + r] * vs[r];
                        sum += x[u][4 * a + r];
                        top = fmaxf(top, w[r]);
                    }
                    pf[u][2 * a] = pack_f16(w[0], w[1]);
                    pf[u][2 * a + 1] = pack_f16(w[2], w[3]);
                }
            if (raise) break;
            raise = __builtin_amdgcn_ballot_w64(!(top <= kMaxP && sum <= kMaxSum)) != 0;
            if (!raise) break;
        }
        l += sum;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int st = 0; st < 4; ++st) {
            const uint32_t *p = &pf[st >> 1][4 * (st & 1)];
            const u32x4 bop = {p[0], p[1], p[2], p[3]};
#pragma unroll
            for (int i = 0; i < DTL; ++i)
                o[i] = mfma32<DT_F16>(lds_get<u32x4>((v_from ^ (32 * st) ^ (64 * (i & 1))) + 4096 * i), bop, o[i]);
        }
    };

    if (t_begin < t_end) {
        Raw raw;
        load(raw, t_begin);
        unpack(raw, lds0 + (t_begin & 1) * Tile::kBytes);
        if (t_begin + 1 < t_end) load(raw, t_begin + 1);
        __syncthreads();
        for (int tile = t_begin; tile < t_end; ++tile) {
            if (tile + 1 < t_end) {
                unpack(raw, lds0 + ((tile + 1) & 1) * Tile::kBytes);
                if (tile + 2 < t_end) load(raw, tile + 2);
            }
            __builtin_amdgcn_sched_barrier(0);
            const int t0 = kPreTile * tile;
            if (t0 < wave_hi && t0 + kPreTile > wave_lo) {
                bool there[4], plain = t0 >= all_lo && t0 + kPreTile <= all_hi;
#pragma unroll
                for (int i = 0; i < 4; ++i) plain = (there[i] = page_of(t0 + 16 * i) >= 0) && plain;
                compute(lds0 + (tile & 1) * Tile::kBytes, t0, there, plain);
            }
            __syncthreads();
        }
    }

    const bool live = w0 + c32 < c0 + ncols;
    const float lsum = pair_sum(l);
    auto put = [&](size_t at, int d, f32x4 v) { *(uint2 *)((uint16_t *)g.out + at + d) = quad_out_bits<DT>(v); };
    auto quad = [&](int i, int a) { return (f32x4){o[i][4 * a], o[i][4 * a + 1], o[i][4 * a + 2], o[i][4 * a + 3]}; };
    if (splits == 1) {
        if (!live) return;
        const float inv = lsum == 0.0f ? 0.0f : 1.0f / lsum;  // (a sum that is not a number shows in the row)
#pragma unroll
        for (int i = 0; i < DTL; ++i)
#pragma unroll
            for (int a = 0; a < 4; ++a) put(row_at, 32 * i + 8 * a + 4 * half, quad(i, a) * inv);
        return;
    }
    // partial sums through the workspace; the last workgroup of the tile to
    // arrive adds them in order, writes and clears
    const size_t tile_at = (size_t)ct * (g.B * g.Hkv) + bh;
    float *part = g.partials + tile_at * g.splits * (size_t)(g.part_cols * ROW);
    const auto rows_at = buf_rsrc(part, (int64_t)splits * g.part_cols * ROW * 4);
    const uint32_t mine = ((32 * wave + c32) * ROW + 4 * half) * 4;  // this lane's quads: + 8 dimensions each
    auto at = [&](int s, int d) { return (int)(mine + (uint32_t)(s * g.part_cols * ROW + d) * 4); };
    auto put_part = [&](int o, f32x4 v) {
        __builtin_amdgcn_raw_buffer_store_b128(bit_as<u32x4>(v), rows_at, o, 0, kPartCoherent);
    };
    auto get_part = [&](int o) { return bit_as<f32x4>(__builtin_amdgcn_raw_buffer_load_b128(rows_at, o, 0, kPartCoherent)); };
    const int ref_at = D - 4 * half;  // (past the sums, for either half)
    if (live) {
#pragma unroll
        for (int q = 0; q < 4 * DTL; ++q) put_part(at(split, 8 * q), quad(q / 4, q % 4));
        if (half == 0) put_part(at(split, ref_at), (f32x4){ref, lsum, 0, 0});
    }
    if (g.apart || !split_tile_last_atomic(g.counters + tile_at, splits)) return;
    if (!live) return;
    // (one split's quads in flight while the one before is added)
    f32x4 now[4 * DTL], next[4 * DTL], rl, rl_next;
    auto fetch = [&](f32x4 (&w)[4 * DTL], f32x4 &r, int s) {
        r = get_part(at(s, ref_at));
#pragma unroll
        for (int q = 0; q < 4 * DTL; ++q) w[q] = get_part(at(s, 8 * q));
    };
    float rr = kNoRef, ll = 0.0f;
#pragma unroll
    for (int i = 0; i < DTL; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;
    fetch(now, rl, 0);
    for (int s = 0; s < splits; ++s) {
        if (s + 1 < splits) fetch(next, rl_next, s + 1);
        const float top = fmaxf(rr, rl[0]);
        const float old = __builtin_amdgcn_exp2f(rr - top), f = __builtin_amdgcn_exp2f(rl[0] - top);
        rr = top;
        ll = ll * old + f * rl[1];
#pragma unroll
        for (int q = 0; q < 4 * DTL; ++q) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int e = 4 * (q % 4) + r;
                o[q / 4][e] = __builtin_fmaf(f, now[q][r], o[q / 4][e] * old);
            }
            now[q] = next[q];
            put_part(at(s, 8 * q), (f32x4){0, 0, 0, 0});
        }
        rl = rl_next;
    }
    const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
#pragma unroll
    for (int i = 0; i < DTL; ++i)
#pragma unroll
        for (int a = 0; a < 4; ++a) put(row_at, 32 * i + 8 * a + 4 * half, quad(i, a) * inv);
    // (both lanes of a row have read its references by now: they run together)
    if (half == 0)
        for (int s = 0; s < splits; ++s) put_part(at(s, ref_at), (f32x4){0, 0, 0, 0});
}

template <int DT, int D>
static hipError_t launch_prefill(const Kv4AttnArgs &g, hipStream_t st) {
    hipLaunchKernelGGL((kv4_prefill_kernel<DT, D>),
                       dim3((unsigned)((int64_t)g.B * g.Hkv * g.col_tiles), (unsigned)g.splits), dim3(64 * kPreWaves), 0,
                       st, g);
    return hipGetLastError();
}

hipError_t launch_kv4_prefill(const Kv4AttnArgs &g, hipStream_t st) {
    if (g.D == 128)
        return g.dtype == DT_BF16 ? launch_prefill<DT_BF16, 128>(g, st) : launch_prefill<DT_F16, 128>(g, st);
    return g.dtype == DT_BF16 ? launch_prefill<DT_BF16, 64>(g, st) : launch_prefill<DT_F16, 64>(g, st);
}

}  // namespace awq4
