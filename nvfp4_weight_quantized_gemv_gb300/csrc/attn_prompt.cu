// attn_prompt.cu -- attention over the paged 8-bit cache for many query rows:
// prompts, chunks of prompts, long verification steps.
//
// The codes go from HBM through shared memory into tcgen05.mma as they are
// stored; nothing of the cache is converted.  What they are multiplied with is
// written as a sum of two E4M3 terms, x = a + b with a = E4M3(x) and
// b = E4M3(x - a): a bf16 query (8 significant bits) is that sum exactly (down
// to 2^-18 of the row's largest entry), a softmax weight to 2^-9 (its second
// term is kept 2^5 larger, under a scale factor of its own, so that this holds
// down to 2^-14 of the largest weight).  Two products at the 8-bit rate cost
// what one would at the 16-bit rate.
//
//   S = (Qa + Qb) K^T             kind::f8f6f4, M = 128 query rows, N = 128 tokens,
//                                 both operands in shared memory, K-major
//   O += (Pa + Pb) V              kind::mxf8f6f4 (a scale for each row and 32 tokens),
//                                 P in tensor memory, V as stored (N-major)
//
// Weights.  With w = s + log2 vscale(page) and W the maximum of w over a row's
// block of 32 tokens, E = ceil(W): the block's weights are 2^(w - E + 8), at
// most 2^8, and its scale factor 2^(E - ref) for the row's reference ref.  So
// each block's weights have E4M3's full range below their own maximum, whatever
// the row's other tokens weigh, a pass over S needs no maximum of the row, and
// O is rescaled only where E exceeds ref by more than 2^40.  The weights' total
// is kept in fp32 from the unrounded weights.
//
// Work split.  A block is 128 query rows (token-major) of one (sequence, kv
// head), a unit 128 tokens of a block's cache, a block's own cost kPOver units
// more; the persistent grid (a CTA an SM) takes equal contiguous ranges, and
// blocks that span several CTAs leave partial results that a second kernel
// joins, in CTA order.  (Joined by the last of the block's CTAs, which has no
// registers left for loads in flight, they took 7 to 20 us; beside the other
// blocks' work, by warps 4-7, they kept those blocks waiting.)
//
// Warps (768 threads), waiting for each other by mbarriers:
//   0, 2   issue S and PV.  A whole warp runs the loop and one elected lane
//          issues: 64 cycles a product of 128 x 128 x 32, the tensor core's
//          rate, where a branch on the lane's number took 165 to 200
//   1      TMA producer: a ring of K tiles and one of V tiles
//   4-7    the next block's queries (E4M3 terms into shared memory) and the
//          finished block's output
//   8-23   softmax, a query row a thread.  A tile's 128 x 128 scores are about
//          1000 instructions for each scheduler, whose latencies one warp does
//          not hide.  Heads of more than 128 entries: all 16 warps work on one
//          tile (four for each 32 tokens), for the shortest time from S to P,
//          which with two S tiles decides.  Others: two groups of eight (four
//          for each 64 tokens), every second tile each, which fill each other's
//          waits, and three S tiles.
// Up to 32 (64) rows of heads of at most 128 entries would leave three quarters (half) of the tile's rows, and
// with them of the softmax warps, without work, while the others' latencies
// decide the time of a tile.  They are put into all quarters (both halves) of the
// tile instead (kCopies), and a copy's warps make the weights of its share of the
// tile's tokens alone (the others' are zero); the output warps add the shares.
// Tensor memory (512 columns): O (DP columns), then S tiles of 128.  A block's
// weights take the place of its own scores: columns [32 k, +8) the first terms
// of token block k, [+8, +16) the second.  Columns [16, 20) and [20, 24) hold their
// scale factors: row 32 c + i has its four in the bytes of column c, lane i, of
// each of the four lane partitions, a byte a token block.  The softmax warps leave
// them in shared memory and tcgen05.cp copies them into all partitions.  V's
// (constant 1) lie in [24, 32).
//
// Measured, calls in a CUDA graph.  A chunk of 2048 tokens over 16384, 24 + 4
// heads of 256: 773 GFLOP in 550 us, 1405 TFLOP/s (0.73 of a large bf16 library
// product), the tensor core busy for two thirds of it.  A prompt of 4096 tokens, 32
// + 8 heads of 128: 137 GFLOP in 183 us, 750 TFLOP/s: a tile's two products take
// 1024 cycles, its 16384 weights about 2300 (15 instructions a weight of a lane,
// schedulers busy for 65 % of it), and a block of 128 rows costs another 6 tiles'
// time for its queries and its output.
//
// The pass over shared prefixes (SharedParams) is the same kernel without masks, a
// group's rows being those of one sequence: the kernel ahead has written where each
// CTA's range begins, blocks that one CTA works on whole leave their part in a
// row's place for the join, and a CTA's first queries, with nothing to hide them, are
// loaded by all softmax warps (3 us for 128 rows of 128).  A tile takes 1.1 us (heads
// of 128) or 1.45 (256).
#include "attn.cuh"
#include "attn_units.h"
#include "tcgen05.cuh"

namespace nvfp4 {

namespace {

constexpr int kPThreads = 768;
constexpr int kPWarps = kPThreads / 32;
constexpr int kPWarpScores = 0, kPWarpProducer = 1, kPWarpProducts = 2, kPWarpEpi = 4, kPWarpSoft = 8, kPSoftWarps = 16;
constexpr int kPBarEpi = 1;                 // named barrier of warps 4-7
constexpr int kPBarAsked = 2;               // of the softmax warps and the producer: the first block's queries are asked for
constexpr uint32_t kPTmemCols = 512;
constexpr uint32_t kPColSfA = 16, kPColSfA2 = 20, kPColSfB = 24;  // of an S tile
constexpr int kPSfBytes = 512;              // scale factors of a tile's first, or second, terms
constexpr int kPSecond = 5;                 // weights' second terms are 2^5 larger
constexpr float kPRefSlack = 40.f;          // a block's exponent above the row's reference
constexpr int kPScaleRing = 8;              // tiles whose page scales are held
constexpr int kPSumStride = 17;             // floats of 16 columns: no bank conflicts

template <int DP>
struct Prm {
    static constexpr int kHalves = DP / 128;
    static constexpr int kQBufs = DP == 128 ? 2 : 1;   // query buffers
    static constexpr int kSBufs = DP == 128 ? 3 : 2;   // S tiles
    static constexpr int kGroups = DP == 128 ? 2 : 1;  // of softmax warps, each with its tiles
    static constexpr int kTiles = DP == 128 ? 4 : 2;   // slots of the K ring and of the V ring
    static constexpr int kSlot = kPTile * DP;          // one K or V tile
    static constexpr int kQ = 2 * kPRows * DP;         // two terms
    static constexpr int kMisc =
        kSBufs * 2 * kPSfBytes + kPScaleRing * 16 * 4 + (2 + 2 + 2 + 16 + 4 * kSBufs) * kPRows * 4 + 2 * DP * 4 + 32 * kTiles + 256;
    static constexpr int kSum = kPRows * (16 + kPSumStride * 4);  // copies' totals, and 16 of their columns
    static constexpr int kBytes = 1024 + kQBufs * kQ + 2 * kTiles * kSlot + kMisc;
    static constexpr int kCopiesBytes = kBytes + kSum;
};

// Instruction descriptors: E4M3 operands (format 0), fp32 accumulator.
// kind::f8f6f4: accumulator format 1 in [4, 6), N >> 3 in [17, 23), M >> 4 in
// [24, 29), both operands K-major.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// kind::mxf8f6f4: B N-major (bit 16), UE8M0 scale factors (bit 23), the first
// byte of B's scale-factor words, byte `sf` of A's (bits [29, 31)).
__host__ __device__ constexpr uint32_t idesc_mxf8(int M, int N, int sf) {
    return (1u << 16) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24) | ((uint32_t)sf << 29);
}
// 32 rows of 16 bytes, back to back -> four columns of each lane partition.  In
// order with the products that the same thread issues.
__device__ __forceinline__ void tmem_copy_sf(uint32_t taddr, uint32_t saddr) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr),
                 "l"(tc::smem_desc_noswizzle(saddr, 0, 128))
                 : "memory");
}
__device__ __forceinline__ void mma_f8_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_mxf8_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], [%1], %2, %3, [%4], [%5], p;\n}\n" ::"r"(
            d),
        "r"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"((uint32_t)accumulate)
        : "memory");
}
// Shared-memory descriptor of an N-major operand in 128-byte swizzled rows
// (a row = one token's 128 entries): `lbo` bytes between groups of 128 entries,
// 1024 bytes between groups of eight tokens.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t lbo) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Two f16x2 -> four E4M3 codes, and back.
__device__ __forceinline__ uint32_t f16x4_e4m3(uint32_t lo, uint32_t hi) {
    uint32_t r;
    asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f16x2 a, %1;\n cvt.rn.satfinite.e4m3x2.f16x2 b, %2;\n"
        " mov.b32 %0, {a, b};\n}\n"
        : "=r"(r)
        : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Four f16 values of at most 2^8 as two terms, the second times 2^kLift.
template <int kLift>
__device__ __forceinline__ void two_terms(uint32_t lo, uint32_t hi, uint32_t &a, uint32_t &b) {
    a = f16x4_e4m3(lo, hi);
    uint32_t x, y;
    e4m3x4_f16(a, x, y);
    x = sub_f16x2(lo, x);
    y = sub_f16x2(hi, y);
    if (kLift) {
        constexpr uint32_t k = (15u + kLift) << 10, kk = k | (k << 16);  // 2^kLift as f16x2
        x = hmul2_u32(x, kk);
        y = hmul2_u32(y, kk);
    }
    b = f16x4_e4m3(x, y);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A (sequence, kv head, block of rows) and where a CTA's range stands in it.
template <int kOver>
struct PrmWalkOf {
    int b, h, rb, tile;
    int t0, q_len, kv_len;
    int tiles;
    long long left;  // units from the block's first to the range's end; its tiles come after kOver of them
    // Units of a head, summed by a warp.
    __device__ static long long head_units(int g, int q_len, int kv_len, int lane) {
        const long long n = prompt_units(g, q_len, kv_len, lane, 32);
        return units_joined(__reduce_add_sync(0xffffffffu, units_low(n)), __reduce_add_sync(0xffffffffu, units_high(n)));
    }
    template <class P>
    __device__ void load(const P &p) {
        attn_sequence(p, b, &t0, &q_len, &kv_len);
    }
    // Tiles of this block in the range.
    __device__ int segment() const { return (int)min((long long)tiles, left - kOver) - tile; }
    // Whether the next block has tiles in the range.
    __device__ bool more() const { return left > tiles + 2 * kOver; }
    // Whether another CTA continues this block.
    __device__ bool cut() const { return left - kOver < tiles; }
    template <class P>
    __device__ void next_block(const P &p) {  // only if more()
        left -= tiles + kOver;
        tile = 0;
        if (++rb * kPRows >= q_len * p.g) {
            rb = 0;
            if (++h == p.c.heads) {
                h = 0;
                do {
                    ++b;
                    load(p);
                } while (q_len == 0);
            }
        }
        tiles = prompt_block_tiles(p.g, q_len, kv_len, rb, attn_causal(p));
    }
};

// The block that begins in a CTA and ends in another one (in the workspace,
// for the kernel that joins its parts).
struct PrmJoin {
    long long ub, U, C;  // its first unit, all units, the CTAs that share them
    int ca, cb;          // its CTAs; cb < ca: there is no such block
    int t0, h, row0, rows;
};

// One for each CTA, after the partial results.
__device__ __forceinline__ PrmJoin *prompt_joins(const AttnParams &p) {
    return reinterpret_cast<PrmJoin *>(p.partials + (size_t)p.ctas * 2 * p.slot_floats);
}

template <int DP, int kCopies, class P>
__global__ void __launch_bounds__(kPThreads, 1)
    attn_prompt_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const P p) {
    constexpr bool kShared = std::is_same<P, SharedParams>::value;
    using PrmWalk = PrmWalkOf<kShared ? kPOverShared : kPOver>;
    using T = Prm<DP>;
    constexpr int kHalves = T::kHalves, kTiles = T::kTiles, kQBufs = T::kQBufs, kSBufs = T::kSBufs, kGroups = T::kGroups;
    constexpr uint32_t kColS = DP;
    extern __shared__ uint8_t smem_dyn[];
    __shared__ long long sh_scan[kPWarps];
    __shared__ PrmWalk sh_walk[2];  // the range's first and last block
    __shared__ uint32_t sh_tmem;
    __shared__ uint64_t sh_bar[kShared ? 25 : 24];
    __shared__ int sh_nan[2];  // by block parity: whether nan_from holds anything
    uint8_t *const smem = smem_dyn + ((1024u - (smem_u32(smem_dyn) & 1023u)) & 1023u);
    uint8_t *const sq = smem;                         // [buffer][term][half][128 rows][128 B], swizzled
    uint8_t *const ring_k = smem + kQBufs * T::kQ;    // [slot][half][128 tokens][128 B], swizzled
    uint8_t *const ring_v = ring_k + kTiles * T::kSlot;
    uint8_t *at = ring_v + kTiles * T::kSlot;
    uint8_t *const ssf = at;                          // [S tile][term][32 lanes][4 quarters of the rows][32 tokens]
    at += kSBufs * 2 * kPSfBytes;
    float *const sscale = reinterpret_cast<float *>(at);       // [ring][2][8]: k scale, log2 of v scale
    at += kPScaleRing * 16 * 4;
    float *const sqs = reinterpret_cast<float *>(at);          // [block parity][row] query scale
    float *const sfin = sqs + 2 * kPRows;                      // [block parity][row] reference after the block
    float *const sref = sfin + 2 * kPRows;                     // [group][row] reference after the group's last tile
    float *const ssum = sref + 2 * kPRows;                     // [block parity][32 tokens][row][2]: weights' total
    float *const semax = ssum + 16 * kPRows;                   // [S tile][32 tokens][row] exponent
    int *const nan_from = reinterpret_cast<int *>(semax + 4 * kSBufs * kPRows);  // [block parity][DP]
    const uint32_t k_full = smem_u32(nan_from + 2 * DP), k_empty = k_full + 8 * kTiles;
    const uint32_t v_full = k_empty + 8 * kTiles, v_empty = v_full + 8 * kTiles;
    const uint32_t bars = smem_u32(sh_bar);
    constexpr int sum_at = T::kBytes - 1024;  // the copies' sums
    // by S tile: scores made, exponents known, weights made, products done
    const uint32_t s_full = bars, e_full = bars + 24, p_full = bars + 48, pv_done = bars + 72;
    // by query buffer: ready and used; accumulator complete and read; by block parity: totals written and read
    const uint32_t q_full = bars + 96, q_free = bars + 112, o_full = bars + 128, o_free = bars + 136;
    const uint32_t st_full = bars + 144, st_free = bars + 160;
    const uint32_t fin = bars + 176;  // by group: the reference after its last tile is settled
    const uint32_t q_first = bars + 192;  // of a pass over prefixes: the first block's queries
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int B = p.n.b;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kTiles; ++s) {
            mbar_init(k_full + 8 * s, 1);
            mbar_init(k_empty + 8 * s, 1);
            mbar_init(v_full + 8 * s, 1);
            mbar_init(v_empty + 8 * s, 1);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(s_full + 8 * i, 2);
            mbar_init(e_full + 8 * i, kPSoftWarps / kGroups);
            mbar_init(p_full + 8 * i, kPSoftWarps / kGroups);
            mbar_init(pv_done + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + 8 * i, 4);
            mbar_init(q_free + 8 * i, 1);
            mbar_init(st_full + 8 * i, kPSoftWarps);
            mbar_init(st_free + 8 * i, 4);
            mbar_init(fin + 8 * i, kPSoftWarps / kGroups);
        }
        sh_nan[0] = sh_nan[1] = 0;
        mbar_init(o_full, 1);
        mbar_init(o_free, 4);
        if (kShared) mbar_init(q_first, kPSoftWarps);
        fence_barrier_init();
    }
    for (int d = threadIdx.x; d < 2 * DP; d += kPThreads) nan_from[d] = 0x7FFFFFFF;
    griddep_wait();
    // Beside this one run the sequences' own tokens.  Not ahead of the wait: that kernel reads the plan's records and the call's
    // inputs without one of its own.
    if (kShared && threadIdx.x == 0) griddep_launch_dependents();
    PrmWalk wk;
    if constexpr (kShared) {  // the kernel ahead has found where this CTA's range begins
        const int4 *const at = reinterpret_cast<const int4 *>(p.walks + blockIdx.x);
        const int4 a = __ldcg(at), b = __ldcg(at + 1);
        wk.b = a.x, wk.h = a.y, wk.rb = a.z, wk.tile = a.w;
        wk.t0 = b.x, wk.q_len = b.y, wk.kv_len = b.z, wk.tiles = b.w;
        wk.left = __ldcg(&p.walks[blockIdx.x].left);
        __syncthreads();  // the barriers, and entries of nan_from
    } else {
        // ---- units of all sequences (a warp sums its share of them), and where this CTA's range begins
        const int chunk = (B + kPWarps - 1) / kPWarps, b0 = warp * chunk, b1 = min(B, b0 + chunk);
        long long mine = 0;
        for (int b = b0; b < b1; ++b) {
            int t0, q_len, kv_len;
            if (!attn_sequence(p, b, &t0, &q_len, &kv_len) && blockIdx.x == 0 && lane == 0)
                atomicOr(p.err, kDevErrAttnInput);
            mine += PrmWalk::head_units(p.g, q_len, kv_len, lane) * p.c.heads;
        }
        if (lane == 0) sh_scan[warp] = mine;
        __syncthreads();
        long long U = 0, before = 0;
        for (int w = 0; w < kPWarps; ++w) {
            if (w < warp) before += sh_scan[w];
            U += sh_scan[w];
        }
        const long long C = min((long long)p.ctas, U);
        PrmJoin *const mine_to_join = prompt_joins(p) + blockIdx.x;
        if (blockIdx.x >= C) {
            if (threadIdx.x == 0) {
                mine_to_join->ca = 0;
                mine_to_join->cb = -1;
            }
            return;
        }
        const long long u0 = blockIdx.x * U / C, u1 = (blockIdx.x + 1) * U / C;
        // The block of unit u, found by the warp that summed its sequence.
        auto locate = [&](long long u, PrmWalk *to) {
            if (u < before || u >= before + mine) return;  // whole warps
            PrmWalk w;
            long long base = before;
            for (w.b = b0;; ++w.b) {
                w.load(p);
                const long long per = PrmWalk::head_units(p.g, w.q_len, w.kv_len, lane);
                if (u < base + per * p.c.heads) {
                    w.h = (int)((u - base) / per);
                    base += w.h * per;
                    break;
                }
                base += per * p.c.heads;
            }
            for (int r = 0;; r += 32) {  // 32 blocks at a time
                const int rb = r + lane;
                const int n = rb * kPRows < w.q_len * p.g ? prompt_block_tiles(p.g, w.q_len, w.kv_len, rb) : 0;
                const int cost = n > 0 ? n + kPOver : 0;
                int incl = cost;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += v;
                }
                const bool here = u >= base + incl - cost && u < base + incl;
                if (__any_sync(0xffffffffu, here)) {
                    if (here) {
                        w.rb = rb;
                        w.tiles = n;
                        w.left = u1 - (base + incl - cost);
                        w.tile = (int)max(0ll, u0 - (base + incl - cost) - kPOver);
                        *to = w;
                    }
                    break;
                }
                base += __shfl_sync(0xffffffffu, incl, 31);
            }
        };
        locate(u0, &sh_walk[0]);
        locate(u1 - 1, &sh_walk[1]);
        __syncthreads();
        wk = sh_walk[0];
        if (threadIdx.x == 0) {
            const PrmWalk &w = sh_walk[1];
            const long long ub = u1 - w.left;
            const bool cut = w.segment() > 0 && w.cut() && ub + kPOver >= u0;
            *mine_to_join = PrmJoin{ub, U, C, (int)blockIdx.x, cut ? (int)(((ub + kPOver + w.tiles) * C - 1) / U) : -1,
                                    w.t0, w.h, w.rb * kPRows, w.q_len * p.g};
        }
    }
    if (wk.segment() <= 0) return;  // a range that ends before its block's first tile
    if (warp == kPWarpScores) {
        tc::tmem_alloc(smem_u32(&sh_tmem), kPTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh_tmem;
    bool dead = false;  // a wait gave up: no more waiting and no more copies; what is computed is void
    auto wait = [&](uint32_t bar, unsigned parity, unsigned what) {
        if (!mbar_try_wait(bar, parity) && !dead && !mbar_wait_bounded(bar, parity)) {
            atomicOr(p.err, what);
            dead = true;
        }
    };
    // Rows from, from + step, .. below `end` (for heads of at most 128 entries these and their neighbours) of block m's
    // queries as two swizzled E4M3 terms, each row scaled by a power of two to a maximum in [2^7, 2^8), by a warp: eight
    // entries a lane, kPar rows of a lane in flight.
    auto load_rows = [&](const PrmWalk &w, int m, int from, int step, int end, auto par, auto asked) {
        constexpr int kPar = decltype(par)::value;
        const int buf = kQBufs == 2 ? m & 1 : 0;
        const int rows = w.q_len * p.g, row0 = w.rb * kPRows;
        const int i0 = row0 / p.g, h0 = row0 - i0 * p.g;  // token and head of the block's first row
        constexpr int kL = DP / 8;  // lanes of a row
        const int sub = lane / kL, l8 = lane % kL * 8;
        auto convert = [&](int r, const uint4 &w8) {
            const int half = l8 >> 7, c = (l8 & 127) >> 4;
            uint8_t *const to = sq + buf * T::kQ + (half * kPRows + r) * 128 + ((c ^ (r & 7)) << 4) + (l8 & 8);
            uint2 first = make_uint2(0, 0), second = first;
            float scale = 0.f;
            if (!kShared || row0 + (r & ~(32 / kL - 1)) < rows) {  // (else these are no rows)
                const uint32_t u[4] = {w8.x, w8.y, w8.z, w8.w};
                // the largest magnitude's bits, and with them its exponent
                const uint32_t two = __vmaxu2(__vmaxu2(u[0] & 0x7FFF7FFFu, u[1] & 0x7FFF7FFFu),
                                              __vmaxu2(u[2] & 0x7FFF7FFFu, u[3] & 0x7FFF7FFFu));
                int most = (int)max(two & 0xFFFFu, two >> 16);
#pragma unroll
                for (int s = kL / 2; s > 0; s >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, s, kL));
                const int e = most > 0 ? min(max((most >> 7) - 127 - 7, -119), 119) : 0;
                const float down = pow2i(-e);
                // a row that is not finite has no scores
                scale = most < 0x7F80 ? pow2i(e) * p.scale_log2 : __int_as_float(0x7FC00000);
                uint32_t h[4], a[2], b[2];
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    h[y] = pack_f16(__uint_as_float(u[y] << 16) * down, __uint_as_float(u[y] & 0xFFFF0000u) * down);
#pragma unroll
                for (int y = 0; y < 2; ++y) two_terms<0>(h[2 * y], h[2 * y + 1], a[y], b[y]);
                first = make_uint2(a[0], a[1]);
                second = make_uint2(b[0], b[1]);
            }
            if (l8 == 0) sqs[(m & 1) * kPRows + r] = scale;
            *reinterpret_cast<uint2 *>(to) = first;
            *reinterpret_cast<uint2 *>(to + kHalves * kPRows * 128) = second;
        };
        for (int r0 = from + sub; r0 < end; r0 += step * kPar) {
            uint4 v[kPar];
#pragma unroll
            for (int z = 0; z < kPar; ++z) {
                const int r = r0 + z * step;
                v[z] = make_uint4(0, 0, 0, 0);
                const int rr = r & (kPRows / kCopies - 1);
                if (row0 + rr < rows && l8 < p.c.d) {
                    const int x = h0 + rr, i = p.g_div(x);
                    const uint16_t *const src =
                        p.q.p + (w.t0 + i0 + i) * p.q.ts + (w.h * p.g + x - i * p.g) * p.q.hs + l8;
                    if (p.q.vec) {
                        v[z] = *reinterpret_cast<const uint4 *>(src);
                    } else {
                        uint32_t *const u = reinterpret_cast<uint32_t *>(&v[z]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) u[e] = (uint32_t)src[2 * e] | ((uint32_t)src[2 * e + 1] << 16);
                    }
                }
            }
            asked();
            if constexpr (kShared) {  // a loop: unrolled, most of its 4 to 8 us were the fetch of its instructions
#pragma unroll 1
                for (int z = 0; z < kPar; ++z) {
                    convert(r0 + z * step, v[0]);
#pragma unroll
                    for (int k = 0; k + 1 < kPar; ++k) v[k] = v[k + 1];
                }
            } else {
#pragma unroll
                for (int z = 0; z < kPar; ++z) convert(r0 + z * step, v[z]);
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
    };
    if (warp == kPWarpProducer) {
        // ------------------------------------------------------------ producer
        const int box = min(p.c.page, 64), boxes = kPTile / box, page_boxes = p.c.page / box;
        const int pages = max(1, kPTile >> p.c.page_log2);      // of a tile
        const uint64_t policy = l2_policy_evict_last();         // other blocks of the head read them too
        fence_proxy_async_global();
        const int i = lane & (boxes - 1), half = lane / boxes;  // this lane's copies
        const uint32_t to = half * kPTile * 128 + i * box * 128;
        int held = -1, held_b = -1, held_h = -1, page = 0;
        float ks = 1.f, lvs = 0.f;
        // Tile n of a ring (of K or V): waits for its slot, then a box a lane.
        auto slot_free = [&](int n, uint32_t empty) {
            if (n >= kTiles) wait(empty + 8 * (n % kTiles), (unsigned)(n / kTiles - 1) & 1u, kDevErrTimeoutEmpty);
            dead = __any_sync(0xffffffffu, dead);
        };
        auto send = [&](int n, const CUtensorMap *map, const uint8_t *ring, uint32_t full, int y, int h, int pgi) {
            const int slot = n % kTiles;
            if (lane == 0 && !dead) mbar_arrive_expect_tx(full + 8 * slot, T::kSlot);
            __syncwarp();
            if (half < kHalves && !dead)
                tma_load_4d(smem_u32(ring) + slot * T::kSlot + to, map, half * 128, y, h, pgi, full + 8 * slot, policy);
        };
        // V follows K by kSBufs - 1 tiles, as their uses do: where those tiles' boxes are
        int v_y[kSBufs - 1], v_h[kSBufs - 1], v_page[kSBufs - 1];
        int j = 0, sent = 0;
        auto send_v = [&](int n) {
            slot_free(n, v_empty);
            send(n, &map_v, ring_v, v_full, v_y[0], v_h[0], v_page[0]);
#pragma unroll
            for (int z = 0; z + 1 < kSBufs - 1; ++z) {
                v_y[z] = v_y[z + 1];
                v_h[z] = v_h[z + 1];
                v_page[z] = v_page[z + 1];
            }
        };
        for (;;) {
            const int seg = wk.segment();
            for (int k = 0; k < seg; ++k, ++j) {
                const int tile = wk.tile + k, pg = tile * kPTile >> p.c.page_log2;
                if (held < 0 || held_b != wk.b || held_h != wk.h || pg < held || pg + pages > held + 32) {
                    // the page numbers and scales of 32 pages, a lane each
                    held = pg;
                    held_b = wk.b;
                    held_h = wk.h;
                    page = p.c.pages;  // beyond the cache: the copy reads zeros
                    ks = 1.f;
                    lvs = 0.f;
                    if (((long long)(pg + lane) << p.c.page_log2) < wk.kv_len) {
                        page = attn_pages(p, wk.b)[pg + lane];
                        if (page < 0 || page >= p.c.pages) {
                            atomicOr(p.err, kDevErrAttnInput);
                            page = p.c.pages;
                        } else {
                            ks = p.c.ks[(size_t)page * p.c.heads + wk.h];
                            lvs = log2f(p.c.vs[(size_t)page * p.c.heads + wk.h]);
                        }
                    }
                    __syncwarp();
                }
                const int src = pg - held;
                const int pgi = __shfl_sync(0xffffffffu, page, src + i / page_boxes);
                const float a = __shfl_sync(0xffffffffu, ks, src + (lane & 7));
                const float c = __shfl_sync(0xffffffffu, lvs, src + (lane & 7));
                // (the first queries are asked for by now: behind two tiles' copies they took 4 us more)
                if (kShared && j == 0) named_barrier(kPBarAsked, kPSoftWarps * 32 + 32);
                // The scales go with K.  Their place in the ring of eight tiles is free: K(j)'s slot was last that
                // of tile j - kTiles, whose scores are made, so the weights of tile j - kTiles - kSBufs are too.
                slot_free(j, k_empty);
                if (lane < pages) {
                    float *const sc = sscale + (j & (kPScaleRing - 1)) * 16;
                    sc[lane] = a;
                    sc[8 + lane] = c;
                }
                __syncwarp();
                const int y = (tile * kPTile + i * box) & (p.c.page - 1);
                send(j, &map_k, ring_k, k_full, y, wk.h, pgi);
                if (j >= kSBufs - 1) send_v(sent++);
                v_y[kSBufs - 2] = y;
                v_h[kSBufs - 2] = wk.h;
                v_page[kSBufs - 2] = pgi;
                if (kSBufs > 2 && j == 0) {  // the first of two
                    v_y[0] = y;
                    v_h[0] = wk.h;
                    v_page[0] = pgi;
                }
            }
            if (!wk.more()) break;
            wk.next_block(p);
        }
        while (sent < j) send_v(sent++);
        // the last copies have landed before the CTA ends
        if (!dead)
            for (int n = max(0, j - kTiles); n < j; ++n)
                if (!mbar_wait_bounded(k_full + 8 * (n % kTiles), (unsigned)(n / kTiles) & 1u) ||
                    !mbar_wait_bounded(v_full + 8 * (n % kTiles), (unsigned)(n / kTiles) & 1u)) {
                    if (lane == 0) atomicOr(p.err, kDevErrTimeoutDrain);
                    break;
                }
    } else if (warp == kPWarpScores) {
        // -------------------------------------------------- S = (Qa + Qb) K^T
        const uint64_t q_desc = tc::smem_desc_sw128(smem_u32(sq), 1024);
        const uint64_t k_desc = tc::smem_desc_sw128(smem_u32(ring_k), 1024);
        int ks = 0, sb = 0;  // slot of the K ring, S tile
        unsigned k_ph = 0, s_ph = 0;
        bool again = false;  // the S tile has been used before
        for (int m = 0;; ++m) {
            const int seg = wk.segment(), buf = kQBufs == 2 ? m & 1 : 0;
            const uint64_t qd = q_desc + (uint32_t)(buf * (T::kQ >> 4));
            wait(q_full + 8 * buf, (unsigned)(m / kQBufs) & 1u, kDevErrTimeoutFull);
            if (kShared && m == 0) wait(q_first, 0, kDevErrTimeoutFull);
            for (int k = 0; k < seg; ++k) {
                wait(k_full + 8 * ks, k_ph, kDevErrTimeoutFull);
                if (again) wait(pv_done + 8 * sb, s_ph ^ 1u, kDevErrTimeoutEmpty);
                __syncwarp();
                tc::fence_after_sync();
                if (elect_one()) {
                    const uint32_t d = tmem + kColS + (uint32_t)sb * kPTile;
                    const uint64_t kd = k_desc + (uint32_t)(ks * (T::kSlot >> 4));
#pragma unroll
                    for (int half = 0; half < kHalves; ++half)
#pragma unroll
                        for (int s = 0; s < 4; ++s)
#pragma unroll
                            for (int term = 0; term < 2; ++term)
                                mma_f8_ss(d, qd + (((term * kHalves + half) * kPRows * 128 + s * 32) >> 4),
                                          kd + ((half * kPTile * 128 + s * 32) >> 4), idesc_f8(kPRows, kPTile),
                                          half + s + term > 0);
                    tc::commit(s_full + 8 * sb);
                    tc::commit(k_empty + 8 * ks);
                    if (k + 1 == seg) tc::commit(q_free + 8 * buf);
                    mbar_arrive(s_full + 8 * sb);  // hands on what came with Q and K
                }
                __syncwarp();
                if (++ks == kTiles) {
                    ks = 0;
                    k_ph ^= 1u;
                }
                if (++sb == kSBufs) {
                    sb = 0;
                    s_ph ^= 1u;
                    again = true;
                }
            }
            if (!wk.more()) break;
            wk.next_block(p);
        }
    } else if (warp == kPWarpProducts) {
        // ------------------------------------------------- O (+)= (Pa + Pb) V
        const uint64_t v_desc = smem_desc_mn_sw128(smem_u32(ring_v), kPTile * 128);
        int vs = 0, sb = 0;
        unsigned v_ph = 0, s_ph = 0;
        for (int m = 0;; ++m) {
            const int seg = wk.segment();
            if (m > 0) wait(o_free, (unsigned)(m - 1) & 1u, kDevErrTimeoutEmpty);
            for (int k = 0; k < seg; ++k) {
                wait(v_full + 8 * vs, v_ph, kDevErrTimeoutFull);
                wait(p_full + 8 * sb, s_ph, kDevErrTimeoutFull);
                __syncwarp();
                tc::fence_after_sync();
                if (elect_one()) {
                    const uint32_t s = tmem + kColS + (uint32_t)sb * kPTile;
                    const uint64_t vd = v_desc + (uint32_t)(vs * (T::kSlot >> 4));
                    const uint32_t sf = smem_u32(ssf) + sb * 2 * kPSfBytes;
                    tmem_copy_sf(s + kPColSfA, sf);
                    tmem_copy_sf(s + kPColSfA2, sf + kPSfBytes);
#pragma unroll
                    for (int blk = 0; blk < 4; ++blk)
#pragma unroll
                        for (int term = 0; term < 2; ++term)
                            mma_mxf8_ts(tmem, s + blk * 32 + term * 8, vd + ((blk * 32 * 128) >> 4),
                                        idesc_mxf8(kPRows, DP, blk), s + (term ? kPColSfA2 : kPColSfA), s + kPColSfB,
                                        k > 0 || blk + term > 0);
                    tc::commit(pv_done + 8 * sb);
                    tc::commit(v_empty + 8 * vs);
                    if (k + 1 == seg) tc::commit(o_full);
                }
                __syncwarp();
                if (++vs == kTiles) {
                    vs = 0;
                    v_ph ^= 1u;
                }
                if (++sb == kSBufs) {
                    sb = 0;
                    s_ph ^= 1u;
                }
            }
            if (!wk.more()) break;
            wk.next_block(p);
        }
    } else if (warp >= kPWarpEpi && warp < kPWarpSoft) {
        // -------------------------------------------------- queries and output
        const int w4 = warp - kPWarpEpi, row = w4 * 32 + lane;
        const uint32_t lanes = (uint32_t)w4 << 21;
        auto load_q = [&](const PrmWalk &w, int m) {  // a warp takes 32 rows
            const int buf = kQBufs == 2 ? m & 1 : 0;
            if (m >= kQBufs) wait(q_free + 8 * buf, (unsigned)(m / kQBufs - 1) & 1u, kDevErrTimeoutEmpty);
            dead = __any_sync(0xffffffffu, dead);
            if (!kShared || m > 0) load_rows(w, m, w4 * 32, 32 / (DP / 8), w4 * 32 + 32, std::integral_constant<int, kShared && DP == 256 ? 8 : 4>(),
                                            [] {});
            if (lane == 0) mbar_arrive(q_full + 8 * buf);
        };
        load_q(wk, 0);
        for (int m = 0;; ++m) {
            const int seg = wk.segment();
            const bool more = wk.more();
            if (more) {
                PrmWalk nx = wk;
                nx.next_block(p);
                load_q(nx, m + 1);
            }
            // ---- block m's output, a row a thread
            const int rows = wk.q_len * p.g, row0 = wk.rb * kPRows, start = attn_start(p, wk.q_len, wk.kv_len);
            const int i0 = row0 / p.g, h0 = row0 - i0 * p.g, i = p.g_div(h0 + row);
            const bool on = row0 + row < rows;
            const int lim = on ? start + i0 + i : -1;
            const int token = wk.t0 + i0 + i, head = wk.h * p.g + h0 + row - i * p.g;
            uint16_t *const yp = p.y + ((size_t)token * p.q.heads + head) * p.c.d;
            const uint16_t *const gp = p.gate.p ? p.gate.p + token * p.gate.ts + head * p.gate.hs : nullptr;
            const int par = m & 1;
            if (kCopies == 1 && gp && on)  // its latency passes while the last tiles are worked on
                for (int c = 0; c < p.c.d; c += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(gp + c));
            wait(st_full + 8 * par, (unsigned)(m >> 1) & 1u, kDevErrTimeoutFull);
            const float ref = sfin[par * kPRows + row];
            float n = -INFINITY, sum = 0.f;
            const float2 *const st = reinterpret_cast<const float2 *>(ssum) + par * 4 * kPRows + row;
#pragma unroll
            for (int q = 0; q < 4; ++q) n = fmaxf(n, st[q * kPRows].x);
            const float nr = n > -INFINITY ? n : 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) sum = fmaf(exp2_approx(st[q * kPRows].x - nr), st[q * kPRows].y, sum);
            const float inv = attn_inverse(n > -INFINITY ? ref - n : 0.f, sum);
            const bool whole = seg == wk.tiles;
            // a part: of the CTA's first block, or of its last, which others continue
            const bool kept = !whole && nvfp4_in_bounds((int)blockIdx.x < p.ctas && (m == 0 || wk.cut()) &&
                                                            4 * kPRows + kPRows * DP <= p.slot_floats,
                                                        p.err);
            float *const part = p.partials + ((size_t)blockIdx.x * 2 + (m == 0 ? 0 : 1)) * p.slot_floats;
            const bool kept_row = kept && (!kShared || on);  // (nobody reads the others)
            if (kCopies == 1 && kept_row) *reinterpret_cast<float4 *>(part + 4 * row) = make_float4(ref, n, sum, 0.f);
            wait(o_full, (unsigned)m & 1u, kDevErrTimeoutFull);
            dead = __any_sync(0xffffffffu, dead);
            tc::fence_after_sync();
            const int *const nf = nan_from + par * DP;
            const bool some_nan = sh_nan[par] != 0;
            const bool gated = gp && on && whole;
            if constexpr (kCopies > 1) {
                // ---- the copies' shares of a row, 16 columns at a time: a thread sums kCols of them
                constexpr int kCopy = kPRows / kCopies, kCols = 16 / kCopies;
                float4 *const totals = reinterpret_cast<float4 *>(smem + sum_at);  // [copy][row]
                float *const sums = reinterpret_cast<float *>(totals + kPRows);     // [copy][row][kPSumStride]
                totals[row] = make_float4(ref, n, sum, 0.f);
                named_barrier(kPBarEpi, 128);
                auto joined = [&](int r) {  // (maxima, total, factor of this thread's copy)
                    float top = -INFINITY, top_n = -INFINITY, all = 0.f;
#pragma unroll
                    for (int q = 0; q < kCopies; ++q) {
                        top = fmaxf(top, totals[q * kCopy + r].x);
                        top_n = fmaxf(top_n, totals[q * kCopy + r].y);
                    }
                    const bool any = top_n > -INFINITY;
#pragma unroll
                    for (int q = 0; q < kCopies; ++q)
                        all = any ? fmaf(exp2_approx(totals[q * kCopy + r].y - top_n), totals[q * kCopy + r].z, all)
                                  : all + totals[q * kCopy + r].z;
                    return make_float4(top, top_n, all, any ? exp2_approx(ref - top) : 1.f);
                };
                const float f = joined(row & (kCopy - 1)).w;
                const int sum_r = row / kCopies, sum_c = row % kCopies * kCols;  // the row and columns that it sums
                const float4 mine = joined(sum_r);
                const float sum_inv = attn_inverse(mine.y > -INFINITY ? mine.x - mine.y : 0.f, mine.z);
                const int sum_lim = sum_r < rows ? start + p.g_div(sum_r) : -1;
                if (kept && sum_c == 0)
                    *reinterpret_cast<float4 *>(part + 4 * sum_r) = make_float4(mine.x, mine.y, mine.z, 0.f);
#pragma unroll 1
                for (int c = 0; c < DP; c += 32) {
                    uint32_t v[32];
                    tmem_ld32(tmem + lanes + c, v);
                    tc::wait_ld();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (c + h > 0) named_barrier(kPBarEpi, 128);  // the columns before have been summed
#pragma unroll
                        for (int z = 0; z < 16; ++z) sums[row * kPSumStride + z] = __uint_as_float(v[16 * h + z]) * f;
                        named_barrier(kPBarEpi, 128);
#pragma unroll
                        for (int k = 0; k < kCols; k += 4) {
                            float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int q = 0; q < kCopies; ++q)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    x[e] += sums[(q * kCopy + sum_r) * kPSumStride + sum_c + k + e];
                            const int d = c + 16 * h + sum_c + k;
                            if (some_nan) {
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (sum_lim >= nf[d + e]) x[e] = __int_as_float(0x7FC00000);
                            }
                            const float4 y = make_float4(x[0], x[1], x[2], x[3]);
                            if (whole)
                                attn_store4(p, wk.t0, wk.h, sum_r, rows, d, y, sum_inv);
                            else if (kept)
                                *reinterpret_cast<float4 *>(part + 4 * kPRows + (d / 4 * kPRows + sum_r) * 4) = y;
                        }
                    }
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < DP; c += 32) {
                    uint32_t v[32];
                    tmem_ld32(tmem + lanes + c, v);
                    uint4 g[4];
                    if (gated && !kShared) {
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            if (c + 8 * z < p.c.d) g[z] = load_rows8(gp + c + 8 * z, p.gate.vec);
                    }
                    tc::wait_ld();
                    if (some_nan) {
#pragma unroll
                        for (int z = 0; z < 32; ++z)
                            if (lim >= nf[c + z]) v[z] = 0x7FC00000u;
                    }
                    if constexpr (kShared) {
                        if (whole && on) {  // a part of its own, as long as a row
                            float *const to = p.rows + ((size_t)token * p.q.heads + head) * (p.c.d + 4);
                            if (c == 0) *reinterpret_cast<float4 *>(to + p.c.d) = make_float4(ref, n, sum, 0.f);
#pragma unroll
                            for (int z = 0; z < 32; z += 4)
                                if (c + z < p.c.d)
                                    *reinterpret_cast<uint4 *>(to + c + z) = make_uint4(v[z], v[z + 1], v[z + 2], v[z + 3]);
                        }
                    }
                    if (whole && !kShared) {
                        if (on) {
#pragma unroll
                            for (int z = 0; z < 4; ++z)
                                if (c + 8 * z < p.c.d) attn_store8(yp + c + 8 * z, gated, g[z], &v[8 * z], inv);
                        }
                    } else if (kept_row) {
#pragma unroll
                        for (int z = 0; z < 32; z += 4)
                            *reinterpret_cast<uint4 *>(part + 4 * kPRows + ((c + z) / 4 * kPRows + row) * 4) =
                                make_uint4(v[z], v[z + 1], v[z + 2], v[z + 3]);
                    }
                }
            }
            tc::fence_before_sync();
            if (some_nan) {  // for the block after the next
                named_barrier(kPBarEpi, 128);
                for (int d = row; d < DP; d += 128) nan_from[par * DP + d] = 0x7FFFFFFF;
                if (row == 0) sh_nan[par] = 0;
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(o_free);
                mbar_arrive(st_free + 8 * par);
            }
            if (!more) break;
            wk.next_block(p);
        }
    } else if (warp >= kPWarpSoft) {
        // ------------------------------------------------------------- softmax
        constexpr int kParts = 4 / kGroups;  // warps for a row of a tile, each with kGroups blocks of 32 tokens
        const int group = (warp - kPWarpSoft) / (kPSoftWarps / kGroups), part = ((warp - kPWarpSoft) >> 2) & (kParts - 1);
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's lanes of tensor memory
        // Its blocks: neighbours, or, of several copies, one that its own copy has (if any) and one that it has not.
        auto block_of = [&](int z) { return kCopies == 1 ? part * kGroups + z : z * kParts + part; };
        int j = 0, sb = 0;  // tile, S tile and its parity
        unsigned s_ph = 0;
        if (kShared) {  // few tiles a CTA: the first block's queries are what they wait for, and these warps have nothing else
            // (each a share of the rows that there are)
            load_rows(wk, 0, (warp - kPWarpSoft) * (32 / (DP / 8)), kPSoftWarps * (32 / (DP / 8)), kPRows,
                      std::integral_constant<int, DP == 128 ? 4 : 8>(),
                      [] { asm volatile("bar.arrive %0, %1;" ::"n"(kPBarAsked), "n"(kPSoftWarps * 32 + 32) : "memory"); });
            if (lane == 0) mbar_arrive(q_first);
        }
        for (int m = 0;; ++m) {
            const int seg = wk.segment(), par = m & 1;
            const int rows = wk.q_len * p.g, row0 = wk.rb * kPRows, start = attn_start(p, wk.q_len, wk.kv_len);
            const int i0 = row0 / p.g, h0 = row0 - i0 * p.g;
            const int all_see = max(0, start + i0 + 1);
            const int some_see = max(0, start + (min(row0 + kPRows, rows) - 1) / p.g + 1);
            const int qrow = row & (kPRows / kCopies - 1);
            const int lim = row0 + qrow < rows ? start + i0 + p.g_div(h0 + qrow) : -1;  // last token that the row sees
            const bool idle = row0 + qrow - lane >= rows;  // no rows in this warp's lanes
            if (m >= 2) wait(st_free + 8 * par, (unsigned)((m >> 1) - 1) & 1u, kDevErrTimeoutEmpty);
            float ref = -INFINITY, nref = -INFINITY, l = 0.f;  // the row's reference: the same in all its threads
            for (int k = 0; k < seg; ++k, ++j) {
                if (kGroups == 2 && (j & 1) != group) {
                    if (++sb == kSBufs) {
                        sb = 0;
                        s_ph ^= 1u;
                    }
                    continue;
                }
                const int tok_t = (wk.tile + k) * kPTile;
                const uint32_t s_tile = tmem + kColS + (uint32_t)(sb * kPTile) + lanes;
                wait(s_full + 8 * sb, s_ph, kDevErrTimeoutFull);
                dead = __any_sync(0xffffffffu, dead);
                tc::fence_after_sync();
                const float *const sc = sscale + (j & (kPScaleRing - 1)) * 16;
                // (a token without a place has no scores, whatever its query holds: no -inf * NaN)
                const float qs = lim < 0 ? 1.f : sqs[par * kPRows + row];
                const bool edge = tok_t + kPTile > all_see;
                float *const em = semax + sb * 4 * kPRows + row;  // [32 tokens][row]
#pragma unroll 1
                for (int z = idle ? kGroups : 0; z < kGroups; ++z) {
                    const int blk = block_of(z), tok = blk * 32;
                    const uint32_t s_col = s_tile + tok;
                    if (blk * kCopies / 4 != (warp & 3) * kCopies / 4) {  // another copy's tokens
                        const uint32_t none[16] = {};
                        tc::st_32x32b_x16(s_col, none);
                        em[blk * kPRows] = -INFINITY;
                        if (z == kGroups - 1) {
                            __syncwarp();
                            if (lane == 0) mbar_arrive(e_full + 8 * sb);
                        }
                        continue;
                    }
                    uint32_t v[32];
                    tmem_ld32(s_col, v);
                    const int pa = tok >> p.c.page_log2, pb = (tok + 16) >> p.c.page_log2;
                    float f0 = sc[pa] * qs, f1 = sc[pb] * qs;
                    f0 = f0 == 0.f ? 1e-38f : f0;  // not -inf * 0 for a token that is not seen
                    f1 = f1 == 0.f ? 1e-38f : f1;
                    const float lv0 = sc[8 + pa], lv1 = sc[8 + pb];
                    tc::wait_ld();
                    if (edge) {
                        const int seen = lim - tok_t - tok;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i > seen) v[i] = 0xFF800000u;
                    }
                    float m0 = __uint_as_float(v[0]), m1 = __uint_as_float(v[16]);
#pragma unroll
                    for (int i = 1; i < 16; ++i) {
                        m0 = fmaxf(m0, __uint_as_float(v[i]));
                        m1 = fmaxf(m1, __uint_as_float(v[16 + i]));
                    }
                    m0 *= f0;
                    m1 *= f1;
                    const float W = fmaxf(m0 + lv0, m1 + lv1), n = fmaxf(m0, m1);
                    if (n > nref + kPRefSlack) {  // the total's own reference
                        l = nref > -INFINITY ? l * exp2_approx(nref - n) : 0.f;
                        nref = n;
                    }
                    const float nr = nref > -INFINITY ? nref : 0.f;
                    const float e = W > -INFINITY ? ceilf(W) : 0.f;
                    em[blk * kPRows] = W > -INFINITY ? e : -INFINITY;
                    if (z == kGroups - 1) {  // the other tokens' exponents are needed later: they pass while weights are made
                        __syncwarp();
                        if (lane == 0) mbar_arrive(e_full + 8 * sb);
                    }
                    const float c0 = lv0 - e + kWeightLift, c1 = lv1 - e + kWeightLift;
                    const bool apart = fabsf(lv0 - lv1) > 32.f;  // two pages whose weights one exponent does not hold
                    if (apart) {
#pragma unroll 1
                        for (int z2 = 0; z2 < 2; ++z2) {
                            const float f = z2 ? f1 : f0;
                            float t = 0.f;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                t += exp2_approx(fmaf(__uint_as_float(z2 ? v[16 + i] : v[i]), f, -nr));
                            l += t;
                        }
                    }
                    const float2 ff0 = make_float2(f0, f0), ff1 = make_float2(f1, f1);
                    const float2 cc0 = make_float2(c0, c0), cc1 = make_float2(c1, c1);
                    float2 s0 = make_float2(0.f, 0.f), s1 = s0;
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 ff = i < 4 ? ff0 : ff1, cc = i < 4 ? cc0 : cc1;
                        float2 x = fma2(make_float2(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1])), ff, cc);
                        float2 y = fma2(make_float2(__uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])), ff, cc);
                        x.x = exp2_approx(x.x);
                        x.y = exp2_approx(x.y);
                        y.x = exp2_approx(y.x);
                        y.y = exp2_approx(y.y);
                        if (i < 4)
                            s0 = add2(s0, add2(x, y));
                        else
                            s1 = add2(s1, add2(x, y));
                        two_terms<kPSecond>(pack_f16(x.x, x.y), pack_f16(y.x, y.y), pk[i], pk[8 + i]);
                    }
                    if (!apart) {
                        // at most 72 where there is a weight; anything where no token is seen (0, not 0 * inf)
                        l = fmaf(s0.x + s0.y, exp2_approx(fminf(-c0 - nr, 126.f)), l);
                        l = fmaf(s1.x + s1.y, exp2_approx(fminf(-c1 - nr, 126.f)), l);
                    }
                    tc::st_32x32b_x16(s_col, pk);
                }
                if (idle) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(e_full + 8 * sb);
                }
                if (edge) {
                    // A zero weight does not hide a NaN: codes that nobody sees become zeros, a NaN that only
                    // some rows see is noted by entry and token (rows see all tokens from one on).
                    const int slot = j % kTiles;
                    wait(v_full + 8 * slot, (unsigned)(j / kTiles) & 1u, kDevErrTimeoutFull);
                    const int at_tok = tok_t + row;
                    uint8_t *const vt = ring_v + slot * T::kSlot + row * 128;
                    if (at_tok >= all_see) {
#pragma unroll 1
                        for (int c = part * (kHalves * 8 / kParts); c < (part + 1) * (kHalves * 8 / kParts); ++c) {
                            uint4 *const at4 = reinterpret_cast<uint4 *>(vt + (c >> 3) * kPTile * 128 + ((c ^ row) & 7) * 16);
                            uint4 w4 = at_tok >= some_see ? make_uint4(0, 0, 0, 0) : *at4;
                            uint32_t *const w = reinterpret_cast<uint32_t *>(&w4);
                            bool changed = at_tok >= some_see;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t bad = ((w[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                                changed |= bad != 0;
                                while (bad) {
                                    const int b = (__ffs(bad) - 1) >> 3;
                                    atomicMin(&nan_from[par * DP + c * 16 + 4 * i + b], at_tok);
                                    sh_nan[par] = 1;
                                    w[i] &= ~(0xFFu << (8 * b));
                                    bad &= bad - 1;
                                }
                            }
                            if (changed) *at4 = w4;
                        }
                    }
                }
                // ---- the row's reference and this block's scale factor
                wait(e_full + 8 * sb, s_ph, kDevErrTimeoutFull);
                const float e_max =
                    idle ? -INFINITY : fmaxf(fmaxf(em[0], em[kPRows]), fmaxf(em[2 * kPRows], em[3 * kPRows]));
                if (kGroups == 2) {
                    // (at a block's first tile too: a group never settles two tiles past one of the other's)
                    if (j > 0) wait(fin + 8 * (group ^ 1), (unsigned)((j - 1) >> 1) & 1u, kDevErrTimeoutFull);
                    ref = k > 0 ? sref[(group ^ 1) * kPRows + row] : -INFINITY;
                }
                const bool raise = ref > -INFINITY && e_max > ref + kPRefSlack;
                if (__any_sync(0xffffffffu, raise)) {
                    // O so far is in units of the old reference; a share of its columns for each four warps
                    wait(pv_done + 8 * (sb ? sb - 1 : kSBufs - 1), sb ? s_ph : s_ph ^ 1u, kDevErrTimeoutFull);
                    dead = __any_sync(0xffffffffu, dead);
                    tc::fence_after_sync();
                    const float f = raise ? exp2_approx(fmaxf(ref - e_max, -126.f)) : 1.f;
                    const uint32_t o = tmem + lanes;
#pragma unroll 1
                    for (int c = part * (DP / kParts); c < (part + 1) * (DP / kParts); c += 32) {
                        uint32_t v[32];
                        tmem_ld32(o + c, v);
                        tc::wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                        tc::st_32x32b_x32(o + c, v);
                    }
                }
                if (raise || ref == -INFINITY) ref = e_max;
                if (kGroups == 2) {
                    if (part == 0) sref[group * kPRows + row] = ref;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(fin + 8 * group);
                }
                if (part == 0 && k + 1 == seg) sfin[par * kPRows + row] = ref;
                const float bias = ref > -INFINITY ? 127.f - ref : 0.f;
#pragma unroll
                for (int z = 0; z < kGroups; ++z) {
                    const int blk = block_of(z);
                    const uint32_t sf = (uint32_t)fminf(fmaxf(em[blk * kPRows] + bias, 0.f), 254.f);
                    uint8_t *const to = ssf + sb * 2 * kPSfBytes + lane * 16 + (warp & 3) * 4 + blk;
                    to[0] = (uint8_t)sf;
                    to[kPSfBytes] = (uint8_t)__vsubus4(sf, kPSecond);
                }
                fence_proxy_async_smem();  // V's codes and the scale factors, for the products
                if (part == 0) {
                    const uint32_t ones[8] = {0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu,
                                              0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu};
                    tmem_st8(s_tile + kPColSfB, ones);
                }
                tc::wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * sb);
                if (++sb == kSBufs) {
                    sb = 0;
                    s_ph ^= 1u;
                }
            }
            reinterpret_cast<float2 *>(ssum)[(par * 4 + group * kParts + part) * kPRows + row] = make_float2(nref, l);
            __syncwarp();
            if (lane == 0) mbar_arrive(st_full + 8 * par);
            if (!wk.more()) break;
            wk.next_block(p);
        }
    }
    // ---- every product has been waited for (o_full) by warps 4-7
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kPWarpScores) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kPTmemCols);
    }
}

// Joins the parts of the block that begins in CTA blockIdx.x of the kernel
// ahead, in CTA order.  The parts are read from L2 with half a part in flight;
// a warp takes eight rows by 16 entries, so that whole sectors are read and
// written.
constexpr int kPJoinThreads = 512;
template <int DP>
__global__ void __launch_bounds__(kPJoinThreads) attn_join_kernel(const AttnParams p) {
    griddep_wait();
    const PrmJoin at = prompt_joins(p)[blockIdx.x];
    if (at.cb < at.ca) return;
    if (!nvfp4_in_bounds(at.ca == (int)blockIdx.x && at.cb < p.ctas && at.C <= p.ctas && at.U >= at.C, p.err)) return;
    const int row = (threadIdx.x >> 5) * 8 + (threadIdx.x & 7), block_row = at.row0 + row;
    if (block_row >= at.rows) return;
    auto stats = [&](int c) {
        return __ldcg(reinterpret_cast<const float4 *>(attn_part(p, c, at.ub, at.U, at.C) + 4 * row));
    };
    constexpr int kPar = DP / 32;  // groups of four entries in flight: half of this thread's
    float4 v[2][kPar];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int z = 0; z < kPar; ++z) v[h][z] = make_float4(0.f, 0.f, 0.f, 0.f);
    // the sums so far in units of 2^top, the weights' total in units of 2^top_n
    float top = -INFINITY, top_n = -INFINITY, total = 0.f;
    for (int c = at.ca; c <= at.cb; ++c) {
        const float *const x =
            attn_part(p, c, at.ub, at.U, at.C) + 4 * kPRows + ((threadIdx.x >> 3 & 3) * kPRows + row) * 4;
        const float4 s = stats(c);
        float4 y[2][kPar];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int z = 0; z < kPar; ++z)
                y[h][z] = __ldcg(reinterpret_cast<const float4 *>(x + (h * kPar + z) * 16 * kPRows));
        const float m = fmaxf(top, s.x), n = fmaxf(top_n, s.y);
        const bool any = n > -INFINITY;
        const float old = any ? exp2_approx(top - m) : 1.f, f = any ? exp2_approx(s.x - m) : 1.f;
        total = any ? fmaf(exp2_approx(s.y - n), s.z, total * exp2_approx(top_n - n)) : total + s.z;
        top = m;
        top_n = n;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int z = 0; z < kPar; ++z) {
                v[h][z].x = fmaf(v[h][z].x, old, f * y[h][z].x);
                v[h][z].y = fmaf(v[h][z].y, old, f * y[h][z].y);
                v[h][z].z = fmaf(v[h][z].z, old, f * y[h][z].z);
                v[h][z].w = fmaf(v[h][z].w, old, f * y[h][z].w);
            }
    }
    const float inv = attn_inverse(top_n > -INFINITY ? top - top_n : 0.f, total);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int z = 0; z < kPar; ++z)
            attn_store4(p, at.t0, at.h, block_row, at.rows, ((threadIdx.x >> 3 & 3) + (h * kPar + z) * 4) * 4, v[h][z],
                        inv);
}

template <int DP, int kCopies, class P>
cudaError_t prompt_launch(const CUtensorMap &k, const CUtensorMap &v, const P &p, cudaStream_t stream) {
    cudaError_t e = launch_behind(attn_prompt_kernel<DP, kCopies, P>, dim3((unsigned)p.ctas), kPThreads,
                                  kCopies > 1 ? Prm<DP>::kCopiesBytes : Prm<DP>::kBytes, stream, k, v, p);
    if (e != cudaSuccess || std::is_same<P, SharedParams>::value) return e;
    return launch_behind(attn_join_kernel<DP>, dim3((unsigned)p.ctas), kPJoinThreads, 0, stream, p);
}

}  // namespace

constexpr int kPrmStaticSmem = 768;

template <int DP, int kCopies, class P = AttnParams>
static cudaError_t prompt_limit(int smem_optin) {
    constexpr int bytes = kCopies > 1 ? Prm<DP>::kCopiesBytes : Prm<DP>::kBytes;
    if (bytes + kPrmStaticSmem > smem_optin) return cudaErrorInvalidValue;
    return cudaFuncSetAttribute(attn_prompt_kernel<DP, kCopies, P>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}
cudaError_t attn_prompt_set_smem_limit(int smem_optin) {
    cudaError_t e = prompt_limit<128, 1>(smem_optin);
    if (e == cudaSuccess) e = prompt_limit<128, 2>(smem_optin);
    if (e == cudaSuccess) e = prompt_limit<128, 4>(smem_optin);
    if (e == cudaSuccess) e = prompt_limit<256, 1>(smem_optin);
    if (e == cudaSuccess) e = prompt_limit<128, 1, SharedParams>(smem_optin);
    return e == cudaSuccess ? prompt_limit<256, 1, SharedParams>(smem_optin) : e;
}

cudaError_t launch_attn_prompt(const CUtensorMap &k, const CUtensorMap &v, const AttnParams &p, cudaStream_t stream) {
    // Heads of more than 128 entries have all softmax warps at one tile, and copies do little (4 kv heads of 256, without
    // and with them: 16 sequences of 8192 tokens 118 and 115 us with 18 rows, 119 and 119 with 60; of 2048 tokens 66 and
    // 60, 68 and 66; of 128 tokens 26 and 29, 28 and 35; one of 16384 tokens 65 and 66, 69 and 71).  8 kv heads of 128:
    // eight sequences of 16384 tokens 82 and 66 us with 24 rows, 85 and 73 with 40; of 300 tokens 20 and 20, of 500 21
    // and 23.
    const int rows = p.n.max_q * p.g;
    return p.c.d > 128  ? prompt_launch<256, 1>(k, v, p, stream)
           : rows <= 32 ? prompt_launch<128, 4>(k, v, p, stream)
           : rows <= 64 ? prompt_launch<128, 2>(k, v, p, stream)
                        : prompt_launch<128, 1>(k, v, p, stream);
}

cudaError_t launch_attn_prompt_pass(const CUtensorMap &k, const CUtensorMap &v, const SharedParams &p, cudaStream_t stream) {
    return p.c.d > 128 ? prompt_launch<256, 1>(k, v, p, stream) : prompt_launch<128, 1>(k, v, p, stream);
}

}  // namespace nvfp4
