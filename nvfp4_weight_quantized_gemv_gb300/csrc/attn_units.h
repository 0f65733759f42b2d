// attn_units.h -- how the attention kernel for prompts counts its work, in
// arithmetic that host and device compile alike.  Not installed.
#pragma once

#ifdef __CUDACC__
#define NVFP4_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define NVFP4_HOST_DEVICE inline
#endif

namespace nvfp4 {

constexpr int kPTile = 128;  // tokens of a unit
constexpr int kPRows = 128;  // query rows of a block
constexpr int kPOver = 6;    // a block's cost besides its tiles, in units (4: 212 us for the prompt, 8: 195)

// Tiles of block `rb` of a sequence's rows: up to the last token that one of them sees.
NVFP4_HOST_DEVICE int prompt_block_tiles(int g, int q_len, int kv_len, int rb) {
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

// The two summands that 32 lanes may add up in 32 bits each, for a lane's n < 2^46.
NVFP4_HOST_DEVICE unsigned units_low(long long n) { return (unsigned)(n & 0xFFFFF); }
NVFP4_HOST_DEVICE unsigned units_high(long long n) { return (unsigned)(n >> 20); }
NVFP4_HOST_DEVICE long long units_joined(unsigned low, unsigned high) { return ((long long)high << 20) + low; }

}  // namespace nvfp4
