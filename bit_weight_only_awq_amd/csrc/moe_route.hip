// moe_route.hip -- mixture-of-experts routing: each token's top experts with
// their softmax weights, and the plan by which products grouped by expert
// (moe.hpp) read their rows.
//
// Choice.  A token's E logits lie in a group of lanes, consecutive experts to a
// lane, as whole-number keys that order as the logits do (an expert that cannot
// be chosen has key 0).  Each of the k rounds takes the largest key of the group
// (a butterfly of moves inside the registers), the lowest lane that holds it and
// that lane's lowest expert -- which is the lower expert of equal logits --
// and takes it out.  Bound by the rounds' chain of dependent moves (about 100
// cycles each), not by memory: a token's wave has 2 E bytes to read.
//
// Plan.  A stable counting sort of the slots t k + j by expert.  Every wave takes
// consecutive slots, 64 at a time: the lanes of one expert find each other by a
// ballot per bit of the expert's number, a lane's place among them is the
// number of such lanes below it, and running counts in LDS (one set a wave) go on
// from group to group.  No atomics whose order could show: the plan is the
// same on every run.
//
// One workgroup does both for few tokens; otherwise a first launch chooses and
// counts, and a second places: its workgroups add up the counts of all others
// for themselves, which for up to 256 of them costs less than a launch between.
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

// The choice of token t by its group of LPT lanes, E <= LPT * PER experts;
// lane j < k of the group writes the j-th.  live: false past the last token (every lane
// takes part in the moves).  ids: LDS, the token's k slots.
template <int LPT, int PER>
__device__ __forceinline__ void choose(const RouteArgs &g, int64_t t, bool live, int16_t *ids) {
    const int lane = threadIdx.x & (LPT - 1);
    const int shift = (threadIdx.x & 63) & ~(LPT - 1);
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane * PER + i;
        key[i] = 0;
        if (live && e < g.E) {
            const size_t at = (size_t)t * g.E + e;
            float l = g.dtype == DT_F16    ? f16_bits_to_f32(((const uint16_t *)g.logits)[at])
                      : g.dtype == DT_BF16 ? bf16_bits_to_f32(((const uint16_t *)g.logits)[at])
                                           : ((const float *)g.logits)[at];
            l += 0.0f;  // -0 and 0 are one logit
            if (l > -__builtin_inff()) {  // (not for NaN)
                l = fminf(l, 3.4028234663852886e38f);
                const uint32_t u = bit_as<uint32_t>(l);
                key[i] = (u & 0x80000000u) ? ~u : u | 0x80000000u;
            }
        }
    }
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) best = max(best, key[i]);
    const uint32_t top = group_max<LPT>(best);
    const float m = top ? key_value(top) : 0.0f;  // no expert: no weight
    float sum = 0.0f;
    if (!g.renormalize) {
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += key[i] ? expf(key_value(key[i]) - m) : 0.0f;
        sum = group_sum<LPT>(sum);
    }
    int my_id = -1;
    float my_w = 0.0f;
    for (int j = 0; j < g.k; ++j) {
        const uint32_t w = j == 0 ? top : group_max<LPT>(best);
        const uint64_t holders = __ballot(best == w) >> shift;
        const int owner = __builtin_ctzll(holders);
        int id = -1;
        if (lane == owner) {
            // this lane's first expert with the key leaves, and its next best comes up
            int at = PER;
#pragma unroll
            for (int i = PER - 1; i >= 0; --i) at = key[i] == w ? i : at;
            id = lane * PER + at;
            best = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (i == at) key[i] = 0;
                best = max(best, key[i]);
            }
        }
        id = __shfl(id, shift + owner, 64);
        const float e = w ? expf(key_value(w) - m) : 0.0f;
        if (g.renormalize) sum += e;
        if (lane == j && w) {
            my_id = id;
            my_w = e;
        }
    }
    if (live && lane < g.k) {
        const size_t at = (size_t)t * g.k + lane;
        g.experts[at] = my_id;
        g.weights[at] = my_id >= 0 ? my_w / sum : 0.0f;
        ids[lane] = (int16_t)my_id;
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

// Counts of the workgroup's slots by wave and expert; run[w][e] is left as the number of the
// expert's slots in waves before w, total[e] as the sum.  id(s): the expert of slot s < n, -1: none.
template <int WAVES, class Id>
__device__ __forceinline__ void count_slots(int n, int E, int bits, int *run, int *total, Id id) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < WAVES * E; i += 64 * WAVES) run[i] = 0;
    __syncthreads();
    const int per = ((n + WAVES - 1) / WAVES + 63) & ~63;
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

// The workgroup's slots to their places: slot s (s0 + s of the call) of expert e to base[e] + its place.
template <int WAVES, class Id>
__device__ __forceinline__ void place_slots(const RouteArgs &g, int64_t s0, int n, int bits, int *run,
                                            const int *base, int live, Id id) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int per = ((n + WAVES - 1) / WAVES + 63) & ~63;
    for (int g0 = wave * per; g0 < min(n, wave * per + per); g0 += 64) {
        const int s = g0 + lane;
        const int e = s < n ? id(s) : -1;
        const int at = take_places(e, bits, run + wave * g.E);
        if (s >= n) continue;
        const int to = e >= 0 ? base[e] + at : -1;
        g.places[s0 + s] = to;
        if (to >= 0) g.rows[to] = (int)(s0 + s);
        if (s0 + s >= live) g.rows[s0 + s] = -1;  // behind the last expert's rows
    }
}

template <int LPT, int PER, int WAVES>
__device__ __forceinline__ void choose_all(const RouteArgs &g, int64_t t0, int tokens, int16_t *ids) {
    constexpr int AT_ONCE = WAVES * (64 / LPT);
    for (int i = 0; i < tokens; i += AT_ONCE) {
        const int mine = i + (int)threadIdx.x / LPT;
        choose<LPT, PER>(g, t0 + mine, mine < tokens, ids + (size_t)mine * g.k);
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
    int16_t *ids = (int16_t *)(all + 1);
    choose_all<LPT, PER, WAVES>(g, 0, (int)g.T, ids);
    const int n = (int)g.T * g.k, bits = expert_bits(g.E);
    auto id = [&](int s) { return (int)ids[s]; };
    count_slots<WAVES>(n, g.E, bits, run, total, id);
    scan_experts(total, g.E, all);
    __syncthreads();
    for (int e = threadIdx.x; e <= g.E; e += 64 * WAVES) g.offsets[e] = e < g.E ? total[e] : *all;
    place_slots<WAVES>(g, 0, n, bits, run, total, *all, id);
}

// First of two launches: choice of the workgroup's tokens, and its slots of each expert to counts[workgroup][e].
template <int LPT, int PER>
__global__ __launch_bounds__(256) void route_choose(RouteArgs g, int block_tokens, int *__restrict__ counts) {
    constexpr int WAVES = 4;
    extern __shared__ int lds[];
    int *total = lds;
    int16_t *ids = (int16_t *)(total + g.E);
    const int64_t t0 = (int64_t)blockIdx.x * block_tokens;
    const int tokens = (int)min((int64_t)block_tokens, g.T - t0);
    for (int e = threadIdx.x; e < g.E; e += 64 * WAVES) total[e] = 0;
    choose_all<LPT, PER, WAVES>(g, t0, tokens, ids);
    for (int s = threadIdx.x; s < tokens * g.k; s += 64 * WAVES)
        if (ids[s] >= 0) atomicAdd(total + ids[s], 1);  // (whole numbers: the order does not show)
    __syncthreads();
    for (int e = threadIdx.x; e < g.E; e += 64 * WAVES) counts[(size_t)blockIdx.x * g.E + e] = total[e];
}

// Second: where each expert begins (the counts of all workgroups), where this workgroup's slots of it
// begin (those before it), and the slots' places.
__global__ __launch_bounds__(256) void route_place(RouteArgs g, int block_tokens, const int *__restrict__ counts) {
    constexpr int WAVES = 4;
    extern __shared__ int lds[];
    int *run = lds, *total = run + WAVES * g.E, *base = total + g.E, *all = base + g.E;
    const int blocks = gridDim.x, me = blockIdx.x, E = g.E;
    const int64_t s0 = (int64_t)me * block_tokens * g.k;
    const int n = (int)min((int64_t)block_tokens * g.k, g.T * g.k - s0);
    const int bits = expert_bits(E);
    const int32_t *mine = g.experts + s0;
    auto id = [&](int s) { return mine[s]; };
    count_slots<WAVES>(n, E, bits, run, total, id);
    for (int e = threadIdx.x; e < E; e += 64 * WAVES) total[e] = base[e] = 0;
    __syncthreads();
    // thread: one expert, every parts-th workgroup
    const int parts = max(1, 64 * WAVES / E);
    for (int i = threadIdx.x; i < E * parts; i += 64 * WAVES) {
        const int e = i % E;
        int sum = 0, before = 0;
        for (int b = i / E; b < blocks; b += 8 * parts) {
            int c[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) c[u] = b + u * parts < blocks ? counts[(size_t)(b + u * parts) * E + e] : 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                sum += c[u];
                before += b + u * parts < me ? c[u] : 0;
            }
        }
        atomicAdd(total + e, sum);
        atomicAdd(base + e, before);
    }
    __syncthreads();
    scan_experts(total, E, all);
    __syncthreads();
    if (me == 0)
        for (int e = threadIdx.x; e <= E; e += 64 * WAVES) g.offsets[e] = e < E ? total[e] : *all;
    for (int e = threadIdx.x; e < E; e += 64 * WAVES) base[e] += total[e];
    __syncthreads();
    place_slots<WAVES>(g, s0, n, bits, run, base, *all, id);
}

template <int LPT, int PER>
static hipError_t launch_route_t(const RouteArgs &g, const RoutePlan &p, hipStream_t st) {
    if (p.blocks == 1) {
        if constexpr (PER <= 8) {  // (the planner gives more experts two launches: their counts would not fit)
            const size_t lds = (size_t)(17 * g.E + 1) * 4 + (size_t)g.T * g.k * 2;
            hipLaunchKernelGGL((route_one<LPT, PER>), dim3(1), dim3(1024), lds, st, g);
            return hipGetLastError();
        }
        return hipErrorInvalidValue;
    }
    const size_t lds = (size_t)g.E * 4 + (size_t)p.block_tokens * g.k * 2;
    hipLaunchKernelGGL((route_choose<LPT, PER>), dim3((unsigned)p.blocks), dim3(256), lds, st, g, p.block_tokens,
                       p.counts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(route_place, dim3((unsigned)p.blocks), dim3(256), (size_t)(6 * g.E + 1) * 4, st, g,
                       p.block_tokens, p.counts);
    return hipGetLastError();
}

hipError_t launch_route(const RouteArgs &g, const RoutePlan &p, hipStream_t st) {
    if (g.E <= 8) return launch_route_t<8, 1>(g, p, st);
    if (g.E <= 16) return launch_route_t<16, 1>(g, p, st);
    if (g.E <= 32) return launch_route_t<32, 1>(g, p, st);
    if (g.E <= 64) return launch_route_t<64, 1>(g, p, st);
    if (g.E <= 128) return launch_route_t<64, 2>(g, p, st);
    if (g.E <= 256) return launch_route_t<64, 4>(g, p, st);
    if (g.E <= 512) return launch_route_t<64, 8>(g, p, st);
    return launch_route_t<64, 16>(g, p, st);
}

// ---------------------------------------------------------------------------
// out[t] = the sum over j, in that order and in fp32, of weights[t][j] times row places[t k + j] of y, rounded
// once.  A thread has 8 columns of a token; its k loads of 16 bytes are in flight together.  Bound by
// memory: each of y's rows is read once, in whole lines.
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
