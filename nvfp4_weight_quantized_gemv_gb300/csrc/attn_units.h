// attn_units.h -- how the attention kernel for prompts counts its work, in
// arithmetic that host and device compile alike.  Not installed.
#pragma once

#include <math.h>

#ifdef __CUDACC__
#define NVFP4_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define NVFP4_HOST_DEVICE inline
#endif

namespace nvfp4 {

constexpr int kPTile = 128;  // tokens of a unit
constexpr int kPRows = 128;  // query rows of a block
constexpr int kPOver = 6;    // a block's cost besides its tiles, in units (4: 212 us for the prompt, 8: 195)
constexpr int kPOverShared = 9;  // that in a pass over shared prefixes, where nothing hides it (4 to 8 us of queries and
                                 // output, 1.1 to 1.5 a tile)

// Tiles of block `rb` of a sequence's rows: up to the last token that one of them sees (all tokens, if not causal).
NVFP4_HOST_DEVICE int prompt_block_tiles(int g, int q_len, int kv_len, int rb, bool causal = true) {
    if (!causal) return kv_len > kPTile ? (kv_len + kPTile - 1) / kPTile : 1;
    const int all = q_len * g, to = (rb + 1) * kPRows;
    const int last = ((to < all ? to : all) - 1) / g;
    const int tiles = (kv_len - q_len + last + kPTile) / kPTile;
    return tiles > 1 ? tiles : 1;
}

// Units of the blocks rb, rb + step, ... of a kv head.  In 64 bits: 3,000,000
// tokens of eight query heads have 2.2e9.
NVFP4_HOST_DEVICE long long prompt_units(int g, int q_len, int kv_len, int rb, int step) {
    long long n = 0;
    for (; rb * kPRows < q_len * g; rb += step) n += prompt_block_tiles(g, q_len, kv_len, rb) + kPOver;
    return n;
}

// The first unit of CTA c, and the CTA of unit u, where C CTAs share U units of a pass over shared prefixes.
constexpr int kSharedMostCtas = 192, kSharedMostUnits = 1 << 24;  // their product is below 2^32
NVFP4_HOST_DEVICE int shared_begin(int c, int U, int C) { return (int)((unsigned)c * (unsigned)U / (unsigned)C); }
NVFP4_HOST_DEVICE int shared_owner(int u, int U, int C) {
    return (int)((((unsigned)u + 1) * (unsigned)C - 1) / (unsigned)U);
}

// Tokens of a chunk of which `least` are wanted (>= 0): whole units, up to the longest sequence's 2^30, where one chunk is all
// of a sequence and needs no more room for its parts than there always is.
constexpr int kChunkUnit = 64;
NVFP4_HOST_DEVICE int shared_chunk(float least) {
    return (int)fminf(ceilf(least * (1.f / kChunkUnit)) + (least == 0.f), 16777216.f) * kChunkUnit;
}

// The two summands that 32 lanes may add up in 32 bits each, for a lane's n < 2^46.
NVFP4_HOST_DEVICE unsigned units_low(long long n) { return (unsigned)(n & 0xFFFFF); }
NVFP4_HOST_DEVICE unsigned units_high(long long n) { return (unsigned)(n >> 20); }
NVFP4_HOST_DEVICE long long units_joined(unsigned low, unsigned high) { return ((long long)high << 20) + low; }

}  // namespace nvfp4
