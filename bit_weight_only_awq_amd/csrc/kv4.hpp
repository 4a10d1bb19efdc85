// kv4.hpp -- the paged key/value cache in 4 bits, as the kernels address it
// (kv4_append.hip writes it; kv4_decode.hip, kv4_attention.hip and
// kv4_prefill.hip read it).
//
// int32 [pages, kv_heads, P (D/4 + 2)]; the words of one page and head:
//   K words  [P][D/8]       AWQ order along the head dimension: nibble i of
//                           word j holds dimension 8j + {0,2,4,6,1,3,5,7}[i]
//   V words  [P/4][D/8][4]  the same words, those of four consecutive tokens
//                           side by side
//   K meta   [P]            scale bits (activation type) | zero point << 16
//   V meta   [P]
// value = (code - zero point) * scale, one scale and zero point per token and
// head.
//
// Why this layout: Q K^T sums over the head dimension, so a lane's matrix-core
// operand is a run of one token's words; P V sums over the tokens, so a lane
// wants one word column of several tokens.  With four tokens' V words side by
// side both are 16-byte loads, and 16 tokens of either are 64 D bytes in one
// run, yet appending a token writes whole words only (no read-modify-write of
// a word that another token shares).
#pragma once

#include "device.hpp"

namespace awq4 {

// 8 or 16 bytes of a buffer: lane offset plus scalar offset.  Cache policy 2,
// non-temporal: a decode step reads a layer's cache once, and the next step
// comes after all the other layers' (64 x 4096-8192 tokens 94 -> 85 us, 2 x
// 131072 63 -> 56 us; caches small enough to stay in the memory-side cache
// from call to call read up to 8 % slower).  Policy 0 for prompts, whose
// workgroups read the same words one after another.
constexpr int kStreamOnce = 2;
template <typename T, int POLICY = kStreamOnce>
__device__ __forceinline__ T buf_get(__amdgpu_buffer_rsrc_t r, uint32_t lane, uint32_t scalar) {
    if constexpr (sizeof(T) == 8)
        return bit_as<T>(__builtin_amdgcn_raw_buffer_load_b64(r, (int)lane, (int)scalar, POLICY));
    else
        return bit_as<T>(__builtin_amdgcn_raw_buffer_load_b128(r, (int)lane, (int)scalar, POLICY));
}

template <int D>
struct Kv4Layout {
    static constexpr int kWords = D / 8;  // packed words of one token and head
    __host__ __device__ static constexpr int head_words(int P) { return P * (D / 4 + 2); }
    __host__ __device__ static constexpr int k_word(int t, int j) { return t * kWords + j; }
    __host__ __device__ static constexpr int v_word(int P, int t, int j) {
        return P * kWords + ((t >> 2) * kWords + j) * 4 + (t & 3);
    }
    __host__ __device__ static constexpr int k_meta(int P, int t) { return 2 * P * kWords + t; }
    __host__ __device__ static constexpr int v_meta(int P, int t) { return 2 * P * kWords + P + t; }
};

}  // namespace awq4
