// moe_route.hip -- mixture-of-experts routing: each token's top experts with
// their softmax weights, and the plan by which products grouped by expert
// (moe.hpp) read their rows.
//
// Choice.  A token's E logits lie in a group of lanes, consecutive experts to a
// lane, as whole-number keys that order as the logits do (an expert that cannot
// be chosen has key 0).  Each of the k rounds takes the largest key of the group
// (a butterfly of moves inside the registers), the lowest lane that holds it and
// that lane's lowest expert -- which is the lower expert of equal logits --
// and takes it out.  Bound by chains of dependent moves and LDS accesses, not by
// memory: a token's wave has 2 E bytes to read.
//
// Plan.  A stable counting sort of the slots t k + j by expert.  Every wave takes
// consecutive slots, 64 at a time: the lanes of one expert find each other by a
// ballot per bit of the expert's number, a lane's place among them is the
// number of such lanes below it, and running counts in LDS (one set a wave) go on
// from group to group.  No atomics whose order could show: the plan is the
// same on every run.
//
// One workgroup does both for few tokens; otherwise a first launch chooses, counts
// and ranks, and a second places: its workgroups add up the counts of all others
// for themselves, which for up to 256 of them costs less than a launch between.  (8191 tokens of 128 experts, top 8: the
// first launch 6.6 us in a graph -- 2.0 of an empty one, 0.8 loads and stores, 0.5 the softmax's sum, 1.8 the eight
// rounds, 1.0 the counts, 0.5 the ranks -- and the second 5.9; one token: 4.9.  More than 256 workgroups there are
// from 2^21 slots on, where it is little beside the rest: 2^19 tokens of 1024 experts, top 32, 2048 workgroups, 6.06 ms, a
// quarter of the tokens 1.33.)
#include "device.hpp"
#include "launch.hpp"

namespace awq4 {

static_assert(kMoeMaxExperts == 64 * 16, "16 experts a lane");

// Largest key of each group of LPT lanes, in all of them.
template <int LPT>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
    auto dpp = [](uint32_t u, auto ctrl) {
        return (uint32_t)__builtin_amdgcn_mov_dpp((int)u, decltype(ctrl)::value, 0xF, 0xF, false);
    };
    v = max(v, dpp(v, std::integral_constant<int, 0xB1>{}));   // lane ^ 1
    v = max(v, dpp(v, std::integral_constant<int, 0x4E>{}));   // lane ^ 2
    v = max(v, dpp(v, std::integral_constant<int, 0x141>{}));  // the other four of eight
    if constexpr (LPT >= 16) v = max(v, dpp(v, std::integral_constant<int, 0x140>{}));  // the other eight of sixteen
    if constexpr (LPT >= 32) {
        const auto q = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = max(q[0], q[1]);
    }
    if constexpr (LPT >= 64) {
        const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = max(h[0], h[1]);
    }
    return v;
}
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
    auto dpp = [](float u, auto ctrl) {
        return bit_as<float>(__builtin_amdgcn_mov_dpp(bit_as<int>(u), decltype(ctrl)::value, 0xF, 0xF, false));
    };
    v += dpp(v, std::integral_constant<int, 0xB1>{});
    v += dpp(v, std::integral_constant<int, 0x4E>{});
    v += dpp(v, std::integral_constant<int, 0x141>{});
    if constexpr (LPT >= 16) v += dpp(v, std::integral_constant<int, 0x140>{});
    if constexpr (LPT >= 32) {
        const auto q = __builtin_amdgcn_permlane16_swap(bit_as<uint32_t>(v), bit_as<uint32_t>(v), false, false);
        v = bit_as<float>(q[0]) + bit_as<float>(q[1]);
    }
    if constexpr (LPT >= 64) {
        const auto h = __builtin_amdgcn_permlane32_swap(bit_as<uint32_t>(v), bit_as<uint32_t>(v), false, false);
        v = bit_as<float>(h[0]) + bit_as<float>(h[1]);
    }
    return v;
}

__device__ __forceinline__ float key_value(uint32_t key) {
    return bit_as<float>((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

// PER logits from element `at` on as fp32, by one or two wide loads where every row allows it.
template <int PER>
__device__ __forceinline__ void load_logits(const RouteArgs &g, size_t at, int have, float (&l)[PER]) {
    struct __attribute__((aligned(PER * 2 < 16 ? PER * 2 : 16))) Halves {
        uint16_t v[PER];
    };
    struct __attribute__((aligned(PER * 4 < 16 ? PER * 4 : 16))) Singles {
        float v[PER];
    };
    const bool wide = g.E % PER == 0;  // (then `at` is a multiple of PER, and the last lane with experts has PER of them)
    if (g.dtype == DT_F32) {
        const float *p = (const float *)g.logits + at;
        if (wide && have > 0) {
            const Singles s = *(const Singles *)p;
#pragma unroll
            for (int i = 0; i < PER; ++i) l[i] = s.v[i];
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) l[i] = i < have ? p[i] : 0.0f;
        }
        return;
    }
    const uint16_t *p = (const uint16_t *)g.logits + at;
    Halves h{};
    if (wide && have > 0) {
        h = *(const Halves *)p;
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) h.v[i] = i < have ? p[i] : 0;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = g.dtype == DT_F16 ? f16_bits_to_f32(h.v[i]) : bf16_bits_to_f32(h.v[i]);
}

// The choice of token t by its group of LPT lanes, E <= LPT * PER experts.  live: false past the last token (every
// lane takes part in the moves).  ids, keys: LDS, the token's k slots; the lane that owns a choice writes it there, and
// the lanes of the group then share the slots.
template <int LPT, int PER>
__device__ __forceinline__ void choose(const RouteArgs &g, int64_t t, bool live, int16_t *ids, uint32_t *keys) {
    const int lane = threadIdx.x & (LPT - 1);
    const int shift = (threadIdx.x & 63) & ~(LPT - 1);
    const int have = live ? min(max(g.E - lane * PER, 0), PER) : 0;
    float l[PER];
    load_logits<PER>(g, (size_t)t * g.E + lane * PER, have, l);
    uint32_t key[PER], best = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        key[i] = 0;
        const float v = l[i] + 0.0f;  // -0 and 0 are one logit
        if (i < have && v > -__builtin_inff()) {  // (not for NaN)
            const uint32_t u = bit_as<uint32_t>(fminf(v, 3.4028234663852886e38f));
            key[i] = (u & 0x80000000u) ? ~u : u | 0x80000000u;
        }
        best = max(best, key[i]);
    }
    const uint32_t top = group_max<LPT>(best);
    const float m = top ? key_value(top) : 0.0f;  // no expert: no weight
    float sum = 0.0f;
    if (!g.renormalize) {
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += key[i] ? expf(key_value(key[i]) - m) : 0.0f;
        sum = group_sum<LPT>(sum);
    }
    for (int j = 0; j < g.k; ++j) {
        const uint32_t w = j == 0 ? top : group_max<LPT>(best);
        const int owner = __builtin_ctzll(__ballot(best == w) >> shift);  // the lowest lane of the group that holds it
        if (lane == owner) {
            // its first expert with the key leaves, and its next best comes up
            int at = 0;
#pragma unroll
            for (int i = PER - 1; i >= 0; --i) at = key[i] == w ? i : at;
            best = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                key[i] = i == at ? 0u : key[i];
                best = max(best, key[i]);
            }
            if (live) {
                ids[j] = (int16_t)(w ? lane * PER + at : -1);
                keys[j] = w;
            }
        }
    }
    __builtin_amdgcn_wave_barrier();  // (LDS accesses of a wave stay in order)
    if (!live) {
        if (g.renormalize) (void)group_sum<LPT>(0.0f);
        return;
    }
    auto weight = [&](int j) { return keys[j] ? expf(key_value(keys[j]) - m) : 0.0f; };
    if (g.renormalize) {
        for (int j = lane; j < g.k; j += LPT) sum += weight(j);
        sum = group_sum<LPT>(sum);
    }
    for (int j = lane; j < g.k; j += LPT) {
        const size_t at = (size_t)t * g.k + j;
        g.experts[at] = ids[j];
        g.weights[at] = ids[j] >= 0 ? weight(j) / sum : 0.0f;
    }
}

// The number of slots of each expert in this wave's 64-slot groups before, `run`
// (LDS, one count an expert and wave), and this group's ids (-1: no expert, and past the end):
// returns the slot's place in the count and moves the counts on.
__device__ __forceinline__ int take_places(int id, int bits, int *run) {
    const int lane = threadIdx.x & 63;
    uint64_t same = __ballot(id >= 0);
    for (int b = 0; b < bits; ++b) {
        const bool one = (id >> b) & 1;
        const uint64_t m = __ballot(one);
        same &= one ? m : ~m;
    }
    const int below = __builtin_popcountll(same & ((1ull << lane) - 1));
    int at = 0;
    if (id >= 0) at = run[id];
    __builtin_amdgcn_wave_barrier();
    if (id >= 0 && below == 0) run[id] = at + __builtin_popcountll(same);
    __builtin_amdgcn_wave_barrier();
    return at + below;
}

// Exclusive sum of total[0 .. E) in place, by the first wave; returns the whole in *all (LDS).
__device__ __forceinline__ void scan_experts(int *total, int E, int *all) {
    if (threadIdx.x >= 64) return;
    const int lane = threadIdx.x, per = (E + 63) >> 6;
    const int e0 = lane * per, e1 = min(E, e0 + per);
    int n = 0;
    for (int e = e0; e < e1; ++e) n += total[e];
    int end = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(end, d, 64);
        if (lane >= d) end += v;
    }
    int at = end - n;
    for (int e = e0; e < e1; ++e) {
        const int c = total[e];
        total[e] = at;
        at += c;
    }
    if (lane == 63) *all = end;
}

// Slots that each wave of a workgroup takes of its n.
template <int WAVES>
__device__ __forceinline__ int slots_per_wave(int n) {
    return ((n + WAVES - 1) / WAVES + 63) & ~63;
}

// Counts of the workgroup's slots by wave and expert; run[w][e] is left as the number of the
// expert's slots in waves before w, total[e] as the sum.  id(s): the expert of slot s < n, -1: none.
template <int WAVES, class Id>
__device__ __forceinline__ void count_slots(int n, int E, int bits, int *run, int *total, Id id) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < WAVES * E; i += 64 * WAVES) run[i] = 0;
    __syncthreads();
    const int per = slots_per_wave<WAVES>(n);
    for (int s0 = wave * per; s0 < min(n, wave * per + per); s0 += 64) {
        const int s = s0 + lane;
        take_places(s < n ? id(s) : -1, bits, run + wave * E);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 64 * WAVES) {
        int at = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const int c = run[w * E + e];
            run[w * E + e] = at;
            at += c;
        }
        total[e] = at;
    }
    __syncthreads();
}

// The slots of the only workgroup to their places: slot s of expert e to base[e] + its place.
template <int WAVES, class Id>
__device__ __forceinline__ void place_slots(const RouteArgs &g, int n, int bits, int *run, const int *base, int live, Id id) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, per = slots_per_wave<WAVES>(n);
    for (int g0 = wave * per; g0 < min(n, wave * per + per); g0 += 64) {
        const int s = g0 + lane;
        const int e = s < n ? id(s) : -1;
        const int at = take_places(e, bits, run + wave * g.E);
        if (s >= n) continue;
        const int to = e >= 0 ? base[e] + at : -1;
        g.places[s] = to;
        if (to >= 0) g.rows[to] = s;
        if (s >= live) g.rows[s] = -1;  // behind the last expert's rows
    }
}

template <int LPT, int PER, int WAVES>
__device__ __forceinline__ void choose_all(const RouteArgs &g, int64_t t0, int tokens, int16_t *ids, uint32_t *keys) {
    constexpr int AT_ONCE = WAVES * (64 / LPT);
    for (int i = 0; i < tokens; i += AT_ONCE) {
        const int mine = i + (int)threadIdx.x / LPT;
        choose<LPT, PER>(g, t0 + mine, mine < tokens, ids + (size_t)mine * g.k, keys + (size_t)mine * g.k);
    }
    __syncthreads();
}

__device__ __forceinline__ int expert_bits(int E) { return 32 - __builtin_clz(E); }

// One launch: choice and plan of all tokens by one workgroup.
template <int LPT, int PER>
__global__ __launch_bounds__(1024) void route_one(RouteArgs g) {
    constexpr int WAVES = 16;
    extern __shared__ int lds[];
    int *run = lds, *total = run + WAVES * g.E, *all = total + g.E;
    uint32_t *keys = (uint32_t *)(all + 1);
    const int n = (int)g.T * g.k;
    int16_t *ids = (int16_t *)(keys + n);
    choose_all<LPT, PER, WAVES>(g, 0, (int)g.T, ids, keys);
    const int bits = expert_bits(g.E);
    auto id = [&](int s) { return (int)ids[s]; };
    count_slots<WAVES>(n, g.E, bits, run, total, id);
    scan_experts(total, g.E, all);
    __syncthreads();
    for (int e = threadIdx.x; e <= g.E; e += 64 * WAVES) g.offsets[e] = e < g.E ? total[e] : *all;
    place_slots<WAVES>(g, n, bits, run, total, *all, id);
}

constexpr int kChooseWaves = 8;

// First of two launches: choice of the workgroup's tokens; each slot's place among the workgroup's of its expert (into
// `places`, for now), and how many it has of each expert, to counts[workgroup][e].
template <int LPT, int PER>
__global__ __launch_bounds__(64 * kChooseWaves) void route_choose(RouteArgs g, int block_tokens, int *__restrict__ counts) {
    constexpr int WAVES = kChooseWaves;
    extern __shared__ int lds[];
    int *run = lds, *total = run + WAVES * g.E;
    uint32_t *keys = (uint32_t *)(total + g.E);
    int16_t *ids = (int16_t *)(keys + block_tokens * g.k);
    const int64_t t0 = (int64_t)blockIdx.x * block_tokens;
    const int tokens = (int)max((int64_t)0, min((int64_t)block_tokens, g.T - t0)), n = tokens * g.k;
    choose_all<LPT, PER, WAVES>(g, t0, tokens, ids, keys);
    const int bits = expert_bits(g.E);
    auto id = [&](int s) { return (int)ids[s]; };
    count_slots<WAVES>(n, g.E, bits, run, total, id);
    for (int e = threadIdx.x; e < g.E; e += 64 * WAVES) counts[(size_t)blockIdx.x * g.E + e] = total[e];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, per = slots_per_wave<WAVES>(n);
    for (int s0 = wave * per; s0 < min(n, wave * per + per); s0 += 64) {
        const int s = s0 + lane;
        const int at = take_places(s < n ? id(s) : -1, bits, run + wave * g.E);
        if (s < n) g.places[t0 * g.k + s] = at;
    }
}

// Second: where each expert begins (the counts of all workgroups), where this workgroup's slots of it
// begin (those before it), and the slots' places.
__global__ __launch_bounds__(1024) void route_place(RouteArgs g, int block_tokens, const int *__restrict__ counts) {
    constexpr int THREADS = 1024;
    extern __shared__ int lds[];
    int *total = lds, *base = total + g.E, *all = base + g.E;
    const int blocks = gridDim.x, me = blockIdx.x, E = g.E;
    const int64_t s0 = (int64_t)me * block_tokens * g.k;
    const int n = (int)min((int64_t)block_tokens * g.k, g.T * g.k - s0);
    int expert = -1, rank = 0;  // of the thread's first slot, on their way while the counts are added up
    if ((int)threadIdx.x < n) {
        expert = g.experts[s0 + threadIdx.x];
        rank = g.places[s0 + threadIdx.x];
    }
    for (int e = threadIdx.x; e < E; e += THREADS) total[e] = base[e] = 0;
    __syncthreads();
    // thread: one expert, every parts-th workgroup
    const int parts = max(1, THREADS / E);
    for (int i = threadIdx.x; i < E * parts; i += THREADS) {
        const int e = i % E;
        int sum = 0, before = 0;
        constexpr int kB = 16;  // loads in flight together
        for (int b = i / E; b < blocks; b += kB * parts) {
            int c[kB];
#pragma unroll
            for (int u = 0; u < kB; ++u) c[u] = b + u * parts < blocks ? counts[(size_t)(b + u * parts) * E + e] : 0;
#pragma unroll
            for (int u = 0; u < kB; ++u) {
                sum += c[u];
                before += b + u * parts < me ? c[u] : 0;
            }
        }
        atomicAdd(total + e, sum);  // (whole numbers: the order does not show)
        atomicAdd(base + e, before);
    }
    __syncthreads();
    scan_experts(total, E, all);
    __syncthreads();
    if (me == 0)
        for (int e = threadIdx.x; e <= E; e += THREADS) g.offsets[e] = e < E ? total[e] : *all;
    const int live = *all;
    for (int i = threadIdx.x; i < n; i += THREADS) {
        const int64_t s = s0 + i;
        if (i >= THREADS) {
            expert = g.experts[s];
            rank = g.places[s];
        }
        const int to = expert >= 0 ? total[expert] + base[expert] + rank : -1;
        g.places[s] = to;
        if (to >= 0) g.rows[to] = (int)s;
        if (s >= live) g.rows[s] = -1;  // behind the last expert's rows
    }
}

// One launch: as many lanes to a token as it has experts for, for the shortest chain.
template <int LPT, int PER>
static hipError_t launch_one(const RouteArgs &g, hipStream_t st) {
    const size_t lds = (size_t)(17 * g.E + 1) * 4 + (size_t)g.T * g.k * 6;
    hipLaunchKernelGGL((route_one<LPT, PER>), dim3(1), dim3(1024), lds, st, g);
    return hipGetLastError();
}
// Two launches: up to eight experts a lane.  A round of choosing costs a wave about 3 instructions an expert of
// its lanes and 12 more, whatever the tokens it has: 8191 tokens of 128 experts take 9.5 us by 64 lanes each and 6 by 16.
template <int LPT, int PER>
static hipError_t launch_two(const RouteArgs &g, const RoutePlan &p, hipStream_t st) {
    const size_t lds = (size_t)(kChooseWaves + 1) * g.E * 4 + (size_t)p.block_tokens * g.k * 6;
    hipLaunchKernelGGL((route_choose<LPT, PER>), dim3((unsigned)p.blocks), dim3(64 * kChooseWaves), lds, st, g,
                       p.block_tokens, p.counts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(route_place, dim3((unsigned)p.blocks), dim3(1024), (size_t)(2 * g.E + 1) * 4, st, g,
                       p.block_tokens, p.counts);
    return hipGetLastError();
}

hipError_t launch_route(const RouteArgs &g, const RoutePlan &p, hipStream_t st) {
    if (p.blocks == 1) {
        if (g.E <= 8) return launch_one<8, 1>(g, st);
        if (g.E <= 16) return launch_one<16, 1>(g, st);
        if (g.E <= 32) return launch_one<32, 1>(g, st);
        if (g.E <= 64) return launch_one<64, 1>(g, st);
        if (g.E <= 128) return launch_one<64, 2>(g, st);
        if (g.E <= 256) return launch_one<64, 4>(g, st);
        if (g.E <= 512) return launch_one<64, 8>(g, st);
        return hipErrorInvalidValue;  // (the planner gives more experts two launches)
    }
    if (g.E <= 8) return launch_two<8, 1>(g, p, st);
    if (g.E <= 16) return launch_two<8, 2>(g, p, st);
    if (g.E <= 32) return launch_two<8, 4>(g, p, st);
    if (g.E <= 64) return launch_two<8, 8>(g, p, st);
    if (g.E <= 128) return launch_two<16, 8>(g, p, st);
    if (g.E <= 256) return launch_two<32, 8>(g, p, st);
    if (g.E <= 512) return launch_two<64, 8>(g, p, st);
    return launch_two<64, 16>(g, p, st);
}

// ---------------------------------------------------------------------------
// out[t] = the sum over j, in that order and in fp32, of weights[t][j] times row places[t k + j] of y, rounded
// once.  A thread has 8 columns of a token; its k loads of 16 bytes are in flight together.  Bound by
// memory: each of y's rows is read once, in whole lines (4095 tokens of eight rows of 4096: 302 MB in 56 us, 5.4 TB/s;
// two rows a token, 64 tokens: 2.6 us, the two dependent loads).
template <int DT, int KB>
__global__ __launch_bounds__(256) void moe_combine(const uint16_t *__restrict__ y, const float *__restrict__ weights,
                                                   const int32_t *__restrict__ places, uint16_t *__restrict__ out,
                                                   int64_t T, int64_t R, int N, int k) {
    const int n = 8 * (blockIdx.x * 256 + threadIdx.x);
    const int64_t t = (int64_t)blockIdx.y + (int64_t)blockIdx.z * 65535;
    if (n >= N || t >= T) return;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += KB) {
        u32x4 v[KB];
        float w[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const int p = j0 + j < k ? places[t * k + j0 + j] : -1;
            const bool have = p >= 0 && p < R;
            w[j] = have ? weights[t * k + j0 + j] : 0.0f;
            v[j] = have ? *(const u32x4 *)(y + (size_t)p * N + n) : (u32x4){0, 0, 0, 0};
        }
#pragma unroll
        for (int j = 0; j < KB; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc[i] = __builtin_fmaf(w[j], act_bits_to_f32<DT>((v[j][i >> 1] >> (16 * (i & 1))) & 0xFFFFu), acc[i]);
    }
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = (uint32_t)f32_to_out_bits(acc[2 * i], DT) | ((uint32_t)f32_to_out_bits(acc[2 * i + 1], DT) << 16);
    *(u32x4 *)(out + (size_t)t * N + n) = o;
}

template <int DT>
static hipError_t launch_combine_t(const CombineArgs &g, hipStream_t st) {
    const dim3 grid((unsigned)((g.N / 8 + 255) / 256), (unsigned)(g.T < 65535 ? g.T : 65535),
                    (unsigned)((g.T + 65534) / 65535));
    auto go = [&](auto kb) {
        hipLaunchKernelGGL((moe_combine<DT, decltype(kb)::value>), grid, dim3(256), 0, st, (const uint16_t *)g.y,
                           g.weights, g.places, (uint16_t *)g.out, g.T, g.R, (int)g.N, g.k);
        return hipGetLastError();
    };
    if (g.k <= 2) return go(std::integral_constant<int, 2>{});
    if (g.k <= 4) return go(std::integral_constant<int, 4>{});
    return go(std::integral_constant<int, 8>{});
}
hipError_t launch_combine(const CombineArgs &g, hipStream_t st) {
    return g.dtype == DT_BF16 ? launch_combine_t<DT_BF16>(g, st) : launch_combine_t<DT_F16>(g, st);
}

}  // namespace awq4
