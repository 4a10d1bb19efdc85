// kv4_prefill.hip -- causal attention over the paged 4-bit cache (layout:
// kv4.hpp, mathematics and masks: kv4_attention.hip) for many query rows per
// key/value head: prompts and chunks of prompts.
//
// Bound: the vector units, which take about 340 instructions for 32 rows and 64
// tokens (an exponential and about four more a score, the rest unpacking and
// addresses), 1500 cycles of a SIMD, beside 1024 of the matrix cores (4 D flops
// a row and token).  So what a token costs is paid once for many rows: a
// workgroup takes 256 rows of a sequence and key/value head (the heads of a
// group side by side, so that they share the unpacking), 32 a wave, and tokens
// go through LDS as 16-bit integers (code - zero point), exact in either
// 16-bit type, 128 a step; each of the eight waves unpacks 16 of them for all.
// Nothing is left of the zero points then, and a score costs one FMA:
//   p_j = 2^(x_j (scale log2(e) s_j) - R),  x_j = q . (c_j - z_j)
// with q as it came (fp16 or bf16 operands by its type); the second product
// is fp16 for both (probabilities with the values' scales, 11 bits; see
// kv4_attention.hip for R).  Transposed 32 x 32 tiles, S^T = K Q^T and O^T =
// V^T P^T: a lane's scores are its own operand of the second product.  V lies
// in LDS by dimension, the tokens of a row in the order in which S^T's rows
// fall to a lane.
//
// The two waves of a SIMD run freely between the barriers, one a step, so that
// one's scores go beside the other's products (the wave with scores goes first:
// 3 us of 168 and of 113; it has the more to issue).  Words are loaded two
// steps ahead and unpacked one ahead, beside the last products with values of a
// step; operands and scales are read from LDS two chunks before their use,
// since what cost most was not work but waiting for LDS (a chunk: a quarter of
// a tile's product, an eighth of its scores).  All of it has to fit the 256
// registers of two waves a SIMD: a single spilled one waits for the cache
// words in flight, which are ahead of it in the queue.
//
// Measured (32 heads over 8, D = 128, bf16): a prompt of 4096 tokens 160 us, 860
// TFLOP/s; five chunks of 700 tokens behind 3000 others with a window of 1000,
// 97 us.  128 rows a workgroup, two of them a CU, a barrier every 64 tokens:
// 225 and 125.  One wave a SIMD with 64 rows: over 600 (the sums alone are 128
// registers, and queries spill).  The two waves of a SIMD made to take turns
// between products and scores by barriers: 223 and 175 (a wave alone issues a
// vector instruction every five cycles, two together one every four).
#include "kv4_ops.hpp"

namespace awq4 {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// Waves of a workgroup (32 rows each), tokens of a tile, and of a step: each
// wave unpacks 16 of its tokens.
constexpr int kPreWaves = 8, kPreTile = 64, kPreStep = 16 * kPreWaves;

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

// LDS, in bytes: for each of four tiles (two steps) keys [64][D] and values
// [D][64] as 16-bit integers, the keys' scales times scale log2(e), the values'
// scales, the logarithms of those as a reference takes them, and the largest
// scale of each run of 16 tokens.  Rows are 128 or 256 bytes, so their 16-byte
// chunks are permuted by the row's number:
// the lanes that an access serves at once read rows one apart and write rows
// one or eight apart.  Chunk c of row r is at row(r) ^ (c << 4): one
// instruction from a per-lane base.
template <int D>
struct PreLds {
    static constexpr uint32_t kSlots = 2 * kPreStep / kPreTile, kTile = 2 * kPreTile * D, kK = 0, kV = kSlots * kTile,
                              kKs = 2 * kV, kVs = kKs + 4 * kSlots * kPreTile, kTo = kVs + 4 * kSlots * kPreTile,
                              kTop = kTo + 4 * kSlots * kPreTile,
                              kBytes = kTop + 16 * kSlots;
    __device__ static uint32_t slot(int tile) { return (uint32_t)tile & (kSlots - 1); }
    __device__ static uint32_t mix(uint32_t r) { return (r ^ (r >> 3)) & 7; }
    __device__ static uint32_t k_row(uint32_t t) { return 2 * D * t + 16 * (D == 128 ? t & 15 : mix(t)); }
    __device__ static uint32_t v_row(uint32_t d) { return 2 * kPreTile * d + 16 * mix(d); }
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

// The largest value of the lanes l, l ^ N, l ^ 2 N, l ^ 3 N (N = 16 or 8).
template <int N>
__device__ __forceinline__ float groups_max(float v) {
    if (N == 16) return column_max(v);
    const int turned = __builtin_amdgcn_update_dpp(0, bit_as<int>(v), 0x128, 0xF, 0xF, false);  // row_ror:8
    const uint32_t c = bit_as<uint32_t>(fmaxf(v, bit_as<float>(turned)));
    const auto q = __builtin_amdgcn_permlane16_swap(c, c, false, false);
    return fmaxf(bit_as<float>((uint32_t)q[0]), bit_as<float>((uint32_t)q[1]));
}

// What a thread holds of its wave's 16 tokens before they are unpacked: a quarter of one
// token's keys, and one word column of four tokens' values.
template <int D>
struct PreKeys {
    typedef uint32_t Words __attribute__((ext_vector_type(D / 32)));
    Words w;
    uint32_t km, vm;  // the token's metas
};
struct PreValues {
    u32x4 w, vm;
};

template <int DT, int D>
__global__ __launch_bounds__(64 * kPreWaves, 1) void kv4_prefill_kernel(Kv4AttnArgs g) {
    using L = Kv4Layout<D>;
    constexpr int COLS = 32 * kPreWaves, KS = D / 16, DTL = D / 32, ROW = D + 4;
    using Lds = PreLds<D>;
    __shared__ __attribute__((aligned(256))) char lds[Lds::kBytes];
    const uint32_t lds0 = lds_address(lds);

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c32 = lane & 31, half = lane >> 5;
    const int ct = g.col_tiles - 1 - (int)(blockIdx.x / (g.B * g.Hkv)), bh = blockIdx.x % (g.B * g.Hkv);
    const int h = bh % g.Hkv, b = bh / g.Hkv, split = blockIdx.y;
    const int G = g.Hq / g.Hkv;

    const Kv4Span<COLS, kPreStep> span(g, b, ct, G);
    const int q0 = span.q0, kv_len = span.kv_len, c0 = span.c0, ncols = span.ncols, splits = span.splits;
    if (ncols <= 0 || split >= splits) return;
    const int t_begin = span.first(split), t_end = span.first(split + 1);
    const int kv_lo = span.kv_lo, kv_hi = span.kv_hi;
    // tokens that all rows of this wave see: [all_lo, all_hi)
    const int w0 = min(c0 + 32 * wave, c0 + ncols - 1), w1 = min(w0 + 32, c0 + ncols);
    const int all_hi = span.pos_of(w0, G) + 1, all_lo = g.window > 0 ? span.pos_of(w1 - 1, G) - g.window + 1 : 0;

    // this lane's row
    const int row = min(c0 + 32 * wave + c32, c0 + ncols - 1), qi = row / G, hg = row - qi * G;
    const int hi = span.pos_of(row, G) + 1, lo = g.window > 0 ? hi - g.window : 0;
    const size_t row_at = ((size_t)(q0 + qi) * g.Hq + h * G + hg) * D;
    u32x4 qf[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) qf[i] = *(const u32x4 *)((const uint16_t *)g.q + row_at + 16 * i + 8 * half);

    const int lgP = __builtin_ctz(g.P);
    const auto *table = (const __attribute__((address_space(4))) int32_t *)(g.tables + (size_t)b * g.table_stride);
    const uint32_t num_pages = (uint32_t)min(g.num_pages, (int64_t)0x7FFFFFFF);
    const uint32_t head_bytes = L::head_words(g.P) * 4, page_bytes = (uint32_t)g.Hkv * head_bytes;
    const char *head = (const char *)g.cache + (size_t)h * head_bytes;
    const int last = max(kv_len - 1, 0) >> lgP;
    auto entry = [&](int t) { return (uint32_t)table[min(t >> lgP, last)]; };
    auto has_page = [&](uint32_t e, int t) { return t < kv_len && e < num_pages; };
    // this wave unpacks tokens 16 wave .. of a step, which are 16 run .. of the
    // tile 2 step + mine: a lane has token lane / 4 and a quarter of its key
    // words, and the value words of tokens 4 vg .. 4 vg + 3 in column vw (D = 64:
    // the upper lanes repeat the lower ones')
    const int run = wave & 3, mine = wave >> 2, kt = lane >> 2, kq = lane & 3;
    const int vw = lane & (L::kWords - 1), vg = (lane / L::kWords) & 3, vn = 4 * run + vg;
    const uint32_t k_at = 4 * L::k_word(kt, (D / 32) * kq), v_at = 4 * L::v_word(g.P, 4 * vg, vw);
    const uint32_t km_at = 4 * L::k_meta(g.P, kt), vm1_at = 4 * L::v_meta(g.P, kt), vm_at = 4 * L::v_meta(g.P, 4 * vg);
    const float score_scale = g.scale * 1.4426950408889634f;
    // (past the last tile these read the last token's page: nothing uses it)
    auto page_at = [&](uint32_t e) {
        return buf_rsrc(head + (uint64_t)(e < num_pages ? e : 0u) * page_bytes, head_bytes);
    };
    auto word_at = [](auto page, uint32_t at, uint32_t scalar) {
        return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(page, (int)at, (int)scalar, 0);
    };
    auto load_keys = [&](PreKeys<D> &r, int tile, uint32_t e) {
        const int t = kPreTile * tile + 16 * run;
        const auto page = page_at(e);
        const uint32_t in = (uint32_t)t & (uint32_t)(g.P - 1);
        r.w = buf_get<typename PreKeys<D>::Words, 0>(page, k_at, in * (4 * L::kWords));
        r.km = word_at(page, km_at, 4 * in);
        r.vm = word_at(page, vm1_at, 4 * in);
    };
    auto load_values = [&](PreValues &r, int tile, uint32_t e) {
        const int t = kPreTile * tile + 16 * run;
        const auto page = page_at(e);
        const uint32_t in = (uint32_t)t & (uint32_t)(g.P - 1);
        r.w = buf_get<u32x4, 0>(page, v_at, in * (4 * L::kWords));
        r.vm = buf_get<u32x4, 0>(page, vm_at, 4 * in);
    };
    // this lane's rows in a buffer: written (key token, value dimension 8 vw,
    // in the chunk of its four tokens) and read (key token, value dimension
    // c32).  Tokens 4 vn .. 4 vn + 3 of a tile are S^T rows of the lanes' half
    // vn & 1, the first or second four by vn & 2, in the 16-token step vn >> 2:
    // that is their chunk of a dimension's row and their place in it.
    const uint32_t k_put = Lds::k_row(16 * run + kt) ^ (16 * (D / 32) * kq);
    const uint32_t v_put = (Lds::v_row(8 * vw) ^ (16 * (2 * (vn >> 2) + (vn & 1)))) + 8 * ((vn >> 1) & 1);
    const uint32_t k_get = Lds::k_row(c32) ^ (16 * half), v_get = Lds::v_row(c32) ^ (16 * half);
    // Tokens that no row sees, or without a page: whatever their metas hold
    // must not reach the sums.
    auto inner = [&](uint32_t e, int t) { return t >= kv_lo && t + 16 <= kv_hi && e < num_pages; };
    // Unpacking, in pieces: the metas of the keys, one word of them; the metas of
    // the values, one column of them.
    auto keys_meta = [&](PreKeys<D> &r, int tile, uint32_t e) {
        const int t = kPreTile * tile + 16 * run;
        if (!inner(e, t)) {
            const bool in = e < num_pages && t + kt >= kv_lo && t + kt < kv_hi;
            r.km = in ? r.km : 0u;
            r.vm = in ? r.vm : 0u;
        }
        if (kq == 0) {
            // a value scale that is not finite moves to the score, as NaN: rows
            // that do not see the token clear the score's exponential, and 0
            // times the scale would bring it back
            const float vs = act_bits_to_f32<DT>(r.vm & 0xFFFFu);
            const uint32_t to = lds0 + Lds::slot(tile) * (4 * kPreTile) + 4 * (16 * run + kt);
            lds_put(to + Lds::kKs, vs - vs == 0.0f ? act_bits_to_f32<DT>(r.km & 0xFFFFu) * score_scale : vs - vs);
            // (2^-90: a p stays in range itself beside scales of next to nothing)
            lds_put(to + Lds::kTo, fmaxf(__builtin_amdgcn_logf(fabsf(vs)) - 5.0f, -90.0f));
        }
        r.km = (r.km >> 16) & 15u;  // the zero point from here on
    };
    auto keys_word = [&](const PreKeys<D> &r, int tile, int i) {
        // word i of the quarter is chunk (D/32) kq + i of the token's row
        const uint32_t w = r.w[i], z = r.km;
        u32x4 o;
        if (DT == DT_F16) {
            const f16x2 s16 = {(f16)0.0625f, (f16)0.0625f};
            const f16x2 zl = bit_as<f16x2>(zconst_f16<0>(z)), zh = bit_as<f16x2>(zconst_f16<1>(z));
            const uint32_t u = w >> 8;
            o[0] = bit_as<uint32_t>(bit_as<f16x2>((w & 0x000F000Fu) | 0x64006400u) + zl);
            o[1] = bit_as<uint32_t>(bit_as<f16x2>((w & 0x00F000F0u) | 0x64006400u) * s16 + zh);
            o[2] = bit_as<uint32_t>(bit_as<f16x2>((u & 0x000F000Fu) | 0x64006400u) + zl);
            o[3] = bit_as<uint32_t>(bit_as<f16x2>((u & 0x00F000F0u) | 0x64006400u) * s16 + zh);
        } else {
            // (integers up to 15 in bf16; the bytes of even hold nibbles 0, 2, 4, 6)
            typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
            const float zf = (float)z;
            const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
            auto two = [&](uint32_t x, int lo8) {
                const f32x2 f = {(float)((x >> lo8) & 0xFFu) - zf, (float)((x >> (lo8 + 16)) & 0xFFu) - zf};
                return bit_as<uint32_t>(__builtin_convertvector(f, bf16x2));
            };
            o = (u32x4){two(even, 0), two(odd, 0), two(even, 8), two(odd, 8)};
        }
        uint32_t to = lds0 + Lds::kK + Lds::slot(tile) * Lds::kTile + k_put;
        asm("" : "+v"(to));
        lds_put(to ^ (16 * i), o);
    };
    auto values_meta = [&](PreValues &r, int tile, uint32_t e) {
        const int t = kPreTile * tile + 16 * run;
        if (!inner(e, t)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = t + 4 * vg + i;
                r.vm[i] = e < num_pages && j >= kv_lo && j < kv_hi ? r.vm[i] : 0u;
            }
        }
        f32x4 f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float vs = act_bits_to_f32<DT>(r.vm[i] & 0xFFFFu);
            f[i] = vs - vs == 0.0f ? vs : 0.0f;
        }
        // the largest scale of the wave's 16 tokens: over the lanes of vg 0 .. 3
        const float top = groups_max<L::kWords>(
            fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3]))));
        if (vw == 0) lds_put(lds0 + Lds::kVs + Lds::slot(tile) * (4 * kPreTile) + 16 * vn, f);
        if (lane == 0) lds_put(lds0 + Lds::kTop + Lds::slot(tile) * 16 + 4 * run, top);
        // the zero points' constants from here on: -(1024 + z) and -(64 + z), two tokens a register
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t zz = perm_b32(r.vm[2 * i + 1], r.vm[2 * i], 0x07060302u) & 0x000F000Fu;
            r.vm[2 * i] = 0xE400E400u | zz;
            r.vm[2 * i + 1] = 0xD400D400u | (zz << 4);
        }
    };
    auto values_column = [&](const PreValues &r, int tile, auto column) {
        constexpr int t8 = decltype(column)::value;
        u32x2 o;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t w = t8 & 1 ? pair_y(r.w[2 * i], r.w[2 * i + 1]) : pair_x(r.w[2 * i], r.w[2 * i + 1]);
            if (col_shift(t8)) w >>= 8;
            const f16x2 s16 = {(f16)0.0625f, (f16)0.0625f};
            if (col_hi(t8))
                o[i] = bit_as<uint32_t>(bit_as<f16x2>((w & 0x00F000F0u) | 0x64006400u) * s16 +
                                        bit_as<f16x2>(r.vm[2 * i + 1]));
            else
                o[i] = bit_as<uint32_t>(bit_as<f16x2>((w & 0x000F000Fu) | 0x64006400u) + bit_as<f16x2>(r.vm[2 * i]));
        }
        // (D = 64: the upper lanes write the lower ones' again)
        uint32_t to = lds0 + Lds::kV + Lds::slot(tile) * Lds::kTile + v_put;
        asm("" : "+v"(to));
        lds_put((to ^ (16 * t8)) + 2 * kPreTile * t8, o);
    };

    f32x16 o[DTL], x[2];
    float ref = kNoRef, l = 0.0f;
    uint32_t pf[2][8];
#pragma unroll
    for (int i = 0; i < DTL; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;

    auto chunk_end = [] { __builtin_amdgcn_sched_barrier(0); };
    // The products of a phase in eight chunks of DTL: four of the values of tile
    // `tile`, each 16 tokens, and four of the keys of the tile after it.  Operands
    // of a chunk are read two chunks ahead.
    auto read_chunk = [&](u32x4 (&a)[DTL], int c, int tile) {
        if (c < 4) {
            uint32_t from = (lds0 + Lds::kV + Lds::slot(tile) * Lds::kTile + v_get) ^ (32 * c);
            asm("" : "+v"(from));
#pragma unroll
            for (int i = 0; i < DTL; ++i) a[i] = lds_get<u32x4>((from ^ (64 * (i & 1))) + 4096 * i);
        } else {
            uint32_t from = lds0 + Lds::kK + Lds::slot(tile + 1) * Lds::kTile + k_get;
            asm("" : "+v"(from));
#pragma unroll
            for (int i = 0; i < DTL; ++i) {
                const int k = (c - 4) * (DTL / 2) + i / 2, u = i % 2;
                a[i] = lds_get<u32x4>((from ^ (32 * k) ^ (D == 64 ? 64 * u : 0)) + 64 * D * u);
            }
        }
    };
    auto do_chunk = [&](const u32x4 (&a)[DTL], int c) {
        if (c == 4) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r) x[u][r] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < DTL; ++i) {
            if (c < 4) {
                const uint32_t *p = &pf[c >> 1][4 * (c & 1)];
                o[i] = mfma32<DT_F16>(a[i], (u32x4){p[0], p[1], p[2], p[3]}, o[i]);
            } else {
                x[i % 2] = mfma32<DT>(a[i], qf[(c - 4) * (DTL / 2) + i / 2], x[i % 2]);
            }
        }
    };
    auto products = [&](int tile, auto first, auto past, auto &&beside) {
        constexpr int from = decltype(first)::value, to = decltype(past)::value;
        u32x4 a[3][DTL];
        read_chunk(a[from % 3], from, tile);
        read_chunk(a[(from + 1) % 3], from + 1, tile);
        chunk_end();
        static_for<to - from>([&](auto n) {
            constexpr int c = from + decltype(n)::value;
            if (c + 2 < to) read_chunk(a[(c + 2) % 3], c + 2, tile);
            do_chunk(a[c % 3], c);
            beside(n);
            chunk_end();
        });
    };
    auto nothing = [](auto) {};

    // Scores to probabilities with scales, x to pf; their sum is added to l.
    // there: the tile's runs of 16 tokens have a page; plain: all of them have,
    // and every row of the wave sees every token.  Where the reference has to be
    // raised, which is rare, the scores are taken again rather than kept.
    auto exponentials = [&](int tile, const bool (&there)[4], bool plain) {
        const int t0 = kPreTile * tile;
        uint32_t ks_from = lds0 + Lds::kKs + Lds::slot(tile) * (4 * kPreTile) + 16 * half;
        constexpr uint32_t kVs = Lds::kVs - Lds::kKs, kTo = Lds::kTo - Lds::kKs;
        asm("" : "+v"(ks_from));  // (so that the reads' offsets stay constants)
        float sum;
        // Chunk c = 4 u + a has the tokens 32 u + 8 a + 4 half + r of the tile, in
        // x[u][4 a + r].  (Opaque where used, so that the 32 comparisons are not kept.)
        const int at = t0 + 4 * half - lo, width = max(hi - lo, 0);
        auto opaque = [](int v) {
            asm volatile("" : "+v"(v));
            return v;
        };
        auto seen = [&](int c, int r, int from) {
            return ((unsigned)(from + 32 * (c / 4) + 8 * (c % 4) + r) < (unsigned)width) & there[c / 2];
        };
        // (the scales of four tokens a chunk, read two chunks ahead)
        f32x4 kr[3], vr[3];
        auto read_scales = [&](int c) {
            kr[c % 3] = lds_get<f32x4>(ks_from + 32 * c);
            vr[c % 3] = lds_get<f32x4>(ks_from + kVs + 32 * c);
        };
        auto numerators = [&](int c, bool masked) {
            const f32x4 ks = kr[c % 3], vs = vr[c % 3];
            float p[4], w[4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                p[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[c / 4][4 * (c % 4) + r], ks[r], -ref));
            if (masked) {
                const int from = opaque(at);
#pragma unroll
                for (int r = 0; r < 4; ++r) p[r] = seen(c, r, from) ? p[r] : 0.0f;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) w[r] = p[r] * vs[r];
            sum = c ? sum + ((p[0] + p[1]) + (p[2] + p[3])) : (p[0] + p[1]) + (p[2] + p[3]);
            pf[c / 4][2 * (c % 4)] = pack_f16(w[0], w[1]);
            pf[c / 4][2 * (c % 4) + 1] = pack_f16(w[2], w[3]);
            // (packed here, not where the branches join: 16 registers less)
            asm("" : "+v"(pf[c / 4][2 * (c % 4)]), "+v"(pf[c / 4][2 * (c % 4) + 1]));
        };
        // The reference: no product of p with its token's scale may pass 2^15;
        // raised, the row's largest is 2^5, which leaves normal fp16 numbers down to
        // 2^-19 of it and an absolute 2^-30 of it below.  A lane's sum of p times the
        // tile's largest scale bounds its products and costs two instructions.  That
        // scale may be of a token that the row does not see, or gives next to no
        // probability, so past the bound the products themselves decide, and the new
        // reference is that of the tokens seen: nothing else costs the row bits.
        // (Raised to 2^9 instead, a window's rows raise theirs so often that the five
        // chunks named above take 130 us.)
        const f32x4 tops = lds_get<f32x4>(lds0 + Lds::kTop + Lds::slot(tile) * 16);
        const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        auto all_numerators = [&](bool masked) {
#pragma unroll
            for (int c = 0; c < 2; ++c) read_scales(c);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                if (c + 2 < 8) read_scales(c + 2);
                chunk_end();
                numerators(c, masked);
                chunk_end();
            }
        };
        __builtin_amdgcn_s_setprio(1);  // (see above)
        if (plain)
            all_numerators(false);
        else
            all_numerators(true);
        bool raise = !(sum * top <= kMaxP && sum <= kMaxSum);
        if (__builtin_amdgcn_ballot_w64(raise) != 0) {
            // (fp16 magnitudes are in the order of their patterns.  From 0x6000, 2^9,
            // not only past 2^15: a row whose sum passes the bound here does so again
            // in the next tiles.)
            typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
            u16x2 most = {0, 0};
#pragma unroll
            for (int i = 0; i < 16; ++i)
                most = __builtin_elementwise_max(most, bit_as<u16x2>(pf[i / 8][i % 8] & 0x7FFF7FFFu));
            raise = !(sum <= kMaxSum) || max(most[0], most[1]) > 0x6000;
        }
        if (__builtin_amdgcn_ballot_w64(raise) != 0) {
            products(tile - 1, std::integral_constant<int, 4>{}, std::integral_constant<int, 8>{}, nothing);
            float m = -__builtin_inff();
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const f32x4 ks = lds_get<f32x4>(ks_from + 32 * c), to = lds_get<f32x4>(ks_from + kTo + 32 * c);
                const int from = opaque(at);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float y = __builtin_fmaf(x[c / 4][4 * (c % 4) + r], ks[r], to[r]);
                    m = seen(c, r, from) ? fmaxf(m, y) : m;
                }
                chunk_end();
            }
            // (rows that need not stay as they are, so that no row's result depends on another's)
            const bool either = pair_max(raise ? 1.0f : 0.0f) != 0.0f;
            m = raised(ref, pair_max(m));
            m = either ? m : ref;
            const float f = __builtin_amdgcn_exp2f(ref - m);
            ref = m;
            l *= f;
#pragma unroll
            for (int i = 0; i < DTL; ++i) o[i] *= f;
            all_numerators(true);
        }
        __builtin_amdgcn_s_setprio(0);
        l += sum;
    };

    if (t_begin < t_end) {
        // Entries of the table are read a tile or more before they are needed
        // (they come through the scalar cache, whose misses are long).
        auto own = [&](int step) { return entry(kPreStep * step + 16 * wave); };
        uint32_t own1 = own(t_begin), own2 = own(t_begin + 1), all[4];
        auto entries = [&](int tile) {
#pragma unroll
            for (int i = 0; i < 4; ++i) all[i] = entry(kPreTile * tile + 16 * i);
        };
        // (the first and the last tile may hold nothing that a row sees)
        const int first = 2 * t_begin + (kPreTile * (2 * t_begin + 1) <= kv_lo);
        entries(first);
        PreKeys<D> keys;
        PreValues values;
        auto unpack_meta = [&](int step) {
            keys_meta(keys, 2 * step + mine, own1);
            values_meta(values, 2 * step + mine, own1);
        };
        auto unpack_piece = [&](int step, auto n) {  // of four
            constexpr int i = decltype(n)::value;
            if (i < D / 32) keys_word(keys, 2 * step + mine, i);
            values_column(values, 2 * step + mine, std::integral_constant<int, 2 * i>{});
            values_column(values, 2 * step + mine, std::integral_constant<int, 2 * i + 1>{});
        };
        using C0 = std::integral_constant<int, 0>;
        using C4 = std::integral_constant<int, 4>;
        using C8 = std::integral_constant<int, 8>;
        auto softmax = [&](int tile) {
            const int t0 = kPreTile * tile;
            bool there[4], plain = t0 >= all_lo && t0 + kPreTile <= all_hi;
#pragma unroll
            for (int i = 0; i < 4; ++i) plain = (there[i] = has_page(all[i], t0 + 16 * i)) && plain;
            exponentials(tile, there, plain);
            entries(tile + 1);
        };
        load_keys(keys, 2 * t_begin + mine, own1);
        load_values(values, 2 * t_begin + mine, own1);
        unpack_meta(t_begin);
        static_for<4>([&](auto n) { unpack_piece(t_begin, n); });
        load_keys(keys, 2 * (t_begin + 1) + mine, own2);
        load_values(values, 2 * (t_begin + 1) + mine, own2);
        own1 = own2;
        own2 = own(t_begin + 2);
        __syncthreads();
        products(first - 1, C4{}, C8{}, nothing);
        for (int step = t_begin; step < t_end; ++step) {
            if (2 * step >= first) {
                softmax(2 * step);
                products(2 * step, C0{}, C8{}, nothing);
            }
            if (step + 1 == t_end) break;
            softmax(2 * step + 1);
            unpack_meta(step + 1);
            products(2 * step + 1, C0{}, C4{}, [&](auto n) { unpack_piece(step + 1, n); });
            load_keys(keys, 2 * (step + 2) + mine, own2);
            load_values(values, 2 * (step + 2) + mine, own2);
            own1 = own2;
            own2 = own(step + 3);
            __syncthreads();
            products(2 * step + 1, C4{}, C8{}, nothing);
        }
        if (kPreTile * (2 * t_end - 1) < kv_hi) {
            softmax(2 * t_end - 1);
            products(2 * t_end - 1, C0{}, C4{}, nothing);
        }
    }

    const bool live = 32 * wave + c32 < ncols;
    auto put = [&](size_t at, int d, f32x4 v) { *(uint2 *)((uint16_t *)g.out + at + d) = quad_out_bits<DT>(v); };
    auto quad = [&](int q) {
        const f32x16 &v = o[q / 4];
        return (f32x4){v[4 * (q % 4)], v[4 * (q % 4) + 1], v[4 * (q % 4) + 2], v[4 * (q % 4) + 3]};
    };
    // (a sum that is not a number shows in the row)
    auto inverse = [&](float sum) {
        sum = ref == kNoRef || fabsf(ref) < kFarRef ? sum : __builtin_nanf("");
        return sum == 0.0f ? 0.0f : 1.0f / sum;
    };
    l = pair_sum(l);
    if (splits == 1) {
        const float inv = inverse(l);
        if (live) {
#pragma unroll
            for (int q = 0; q < 4 * DTL; ++q) put(row_at, 8 * q + 4 * half, quad(q) * inv);
        }
        return;
    }
    // partial sums through the workspace, which a second kernel adds
    if (!live) return;
    float *part = g.partials + ((((size_t)ct * (g.B * g.Hkv) + bh) * g.splits + split) * g.part_cols + 32 * wave + c32) * ROW;
#pragma unroll
    for (int q = 0; q < 4 * DTL; ++q) *(f32x4 *)(part + 8 * q + 4 * half) = quad(q);
    if (half == 0) *(f32x4 *)(part + D) = (f32x4){ref, l, 0, 0};
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
