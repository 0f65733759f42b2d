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
// head), a unit 128 tokens of a block's cache; the persistent grid (a CTA an
// SM) takes equal contiguous ranges of the units, and blocks that span several
// CTAs are joined in CTA order as in the kernel for few rows.
//
// Warps (384 threads):
//   0-3, 4-7  softmax of every second tile, a query row a thread; then the next
//             block's queries and the finished block's output
//   8         TMA producer: a ring of K and V tiles in the order of their use
//             (K0 K1 V0 K2 V1 ...)
//   9         MMA issuer: S(i + 1) is issued before PV(i), so that the tensor
//             core works on it while tile i's weights are made
// Tensor memory (512 columns): O in [0, 256), two S tiles of 128 columns.  A
// block's weights take the place of its own scores: columns [32 k, +8) the
// first terms of token block k, [+8, +16) the second; the scale factors of P
// and (constant 1) V lie in what is left of block 0.
#include "attn.cuh"
#include "tcgen05.cuh"

namespace nvfp4 {

namespace {

constexpr int kPTile = 128;                 // tokens of a unit
constexpr int kPRows = 128;                 // query rows of a block
constexpr int kPSoftWarps = 8;
constexpr int kPSoft = kPSoftWarps * 32;
constexpr int kPThreads = 384;
constexpr int kPWarpProducer = 8, kPWarpMma = 9;
constexpr int kPBarSoft = 1;                // named barrier of the softmax warps
constexpr uint32_t kPTmemCols = 512;
constexpr uint32_t kPColS = 256;            // S tiles: columns 256 and 384
constexpr uint32_t kPColSfA = 16, kPColSfA2 = 20, kPColSfB = 24;  // within an S tile
constexpr int kPSecond = 5;                 // weights' second terms are 2^5 larger
constexpr float kPRefSlack = 40.f;          // a block's exponent above the row's reference
constexpr int kPScaleRing = 8;              // tiles whose page scales are held

template <int DP>
struct Prm {
    static constexpr int kHalves = DP / 128;
    static constexpr int kSlot = kPTile * DP;          // one K or V tile
    static constexpr int kSlots = DP == 256 ? 4 : 8;
    static constexpr int kQ = 2 * kPRows * DP;         // two terms
    static constexpr int kMisc = kPScaleRing * 16 * 4 + kPRows * (1 + 4) * 4 + DP * 4 + 16 * kSlots + 256;
    static constexpr int kBytes = 1024 + kQ + kSlots * kSlot + kMisc;
};

// Instruction descriptors: E4M3 operands (format 0), fp32 accumulator.
// kind::f8f6f4: accumulator format 1 in [4, 6), N >> 3 in [17, 23), M >> 4 in
// [24, 29), both operands K-major.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// kind::mxf8f6f4: B N-major (bit 16), UE8M0 scale factors (bit 23), the byte of
// the scale-factor word in [4, 6) for B and [29, 31) for A.
__host__ __device__ constexpr uint32_t idesc_mxf8(int M, int N, int byte) {
    return ((uint32_t)byte << 4) | (1u << 16) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24) |
           ((uint32_t)byte << 29);
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
__device__ __forceinline__ void tmem_st1(uint32_t taddr, uint32_t v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v) : "memory");
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
struct PrmWalk {
    int b, h, rb, tile;
    int t0, q_len, kv_len;
    int tiles;
    long long first;
    __device__ static int block_tiles(int g, int q_len, int kv_len, int rb) {
        const int last = (min((rb + 1) * kPRows, q_len * g) - 1) / g;
        return max(1, (kv_len - q_len + last + kPTile) / kPTile);
    }
    // Units of a head, summed by a warp.
    __device__ static long long head_units(int g, int q_len, int kv_len, int lane) {
        int n = 0;
        for (int rb = lane; rb * kPRows < q_len * g; rb += 32) n += block_tiles(g, q_len, kv_len, rb);
        return __reduce_add_sync(0xffffffffu, n);
    }
    __device__ void load(const AttnParams &p) { kv_sequence(p.n, b, &t0, &q_len, &kv_len); }
    __device__ void next_block(const AttnParams &p) {  // only while units are left
        first += tiles;
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
        tiles = block_tiles(p.g, q_len, kv_len, rb);
    }
};

template <int DP>
__global__ void __launch_bounds__(kPThreads, 1)
    attn_prompt_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                       const AttnParams p) {
    using T = Prm<DP>;
    constexpr int kHalves = T::kHalves, kSlots = T::kSlots;
    extern __shared__ uint8_t smem_dyn[];
    __shared__ long long sh_scan[kPThreads / 32];
    __shared__ PrmWalk sh_walk;
    __shared__ uint32_t sh_tmem;
    __shared__ int sh_last;
    __shared__ uint64_t sh_bar[16];
    uint8_t *const smem = smem_dyn + ((1024u - (smem_u32(smem_dyn) & 1023u)) & 1023u);
    uint8_t *const sq = smem;                      // [term][half][128 rows][128 B], swizzled
    uint8_t *const ring = smem + T::kQ;            // [slot][half][128 tokens][128 B], swizzled
    uint8_t *at = ring + kSlots * T::kSlot;
    float *const sscale = reinterpret_cast<float *>(at);   // [ring][2][8]: k scale, log2 of v scale
    at += kPScaleRing * 16 * 4;
    float *const sref = reinterpret_cast<float *>(at);     // [row] reference exponent
    float *const ssum = sref + kPRows;                     // [wg][row][2]: reference and total of the weights
    int *const nan_from = reinterpret_cast<int *>(ssum + 4 * kPRows);  // [DP]
    const uint32_t full = smem_u32(nan_from + DP), empty = full + 8 * kSlots;
    const uint32_t bars = smem_u32(sh_bar);
    const uint32_t s_full = bars, p_full = bars + 16, fin = bars + 32, pv_done = bars + 48;  // [2] each, by tile parity
    const uint32_t q_full = bars + 64, o_full = bars + 72, o_free = bars + 80;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int B = p.n.b;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + 8 * i, 2);
            mbar_init(p_full + 8 * i, 4);
            mbar_init(fin + 8 * i, 4);
            mbar_init(pv_done + 8 * i, 1);
        }
        mbar_init(q_full, kPSoftWarps);
        mbar_init(o_full, 1);
        mbar_init(o_free, kPSoftWarps);
        fence_barrier_init();
    }
    // ---- units of all sequences (a warp sums its share of them), and where this CTA's range begins
    const int chunk = (B + kPThreads / 32 - 1) / (kPThreads / 32), b0 = warp * chunk, b1 = min(B, b0 + chunk);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
        int t0, q_len, kv_len;
        if (!kv_sequence(p.n, b, &t0, &q_len, &kv_len) && blockIdx.x == 0 && lane == 0)
            atomicOr(p.err, kDevErrAttnInput);
        mine += PrmWalk::head_units(p.g, q_len, kv_len, lane) * p.c.heads;
    }
    if (lane == 0) sh_scan[warp] = mine;
    __syncthreads();
    long long U = 0, before = 0;
    for (int w = 0; w < kPThreads / 32; ++w) {
        if (w < warp) before += sh_scan[w];
        U += sh_scan[w];
    }
    const long long C = min((long long)p.ctas, U);
    if (blockIdx.x >= C) return;
    const long long u0 = blockIdx.x * U / C, u1 = (blockIdx.x + 1) * U / C;
    if (u0 >= before && u0 < before + mine) {  // whole warps
        PrmWalk w;
        long long base = before;
        for (w.b = b0;; ++w.b) {
            w.load(p);
            const long long per = PrmWalk::head_units(p.g, w.q_len, w.kv_len, lane);
            if (u0 < base + per * p.c.heads) {
                w.h = (int)((u0 - base) / per);
                base += w.h * per;
                break;
            }
            base += per * p.c.heads;
        }
        // the block: 32 at a time
        for (int r = 0;; r += 32) {
            const int rb = r + lane;
            const int n = rb * kPRows < w.q_len * p.g ? PrmWalk::block_tiles(p.g, w.q_len, w.kv_len, rb) : 0;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            const bool here = u0 >= base + incl - n && u0 < base + incl;
            if (__any_sync(0xffffffffu, here)) {
                if (here) {
                    w.rb = rb;
                    w.tiles = n;
                    w.first = base + incl - n;
                    w.tile = (int)(u0 - w.first);
                    sh_walk = w;
                }
                break;
            }
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    if (warp == kPWarpMma) {
        tc::tmem_alloc(smem_u32(&sh_tmem), kPTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh_tmem;
    PrmWalk wk = sh_walk;
    bool dead = false;  // a wait gave up: no more waiting, no more copies or products
    auto wait = [&](uint32_t bar, unsigned parity, unsigned what) {
        if (!dead && !mbar_wait_bounded(bar, parity)) {
            atomicOr(p.err, what);
            dead = true;
        }
    };

    if (warp == kPWarpProducer) {
        // ------------------------------------------------------------ producer
        const int box = min(p.c.page, 64), boxes = kPTile / box, page_boxes = p.c.page / box;
        const int pages = max(1, kPTile >> p.c.page_log2);  // of a tile
        const uint64_t policy = l2_policy_evict_last();     // other blocks of the head read them too
        int slot = 0;
        unsigned ph = 0;
        long long item = 0;
        int held = -1, held_b = -1, held_h = -1, page = 0;
        float ks = 1.f, lvs = 0.f;
        // the page numbers and scales of 32 pages from the first one of tile `from`, a lane each
        auto hold = [&](int from, int tile) {
            const int a = from * kPTile >> p.c.page_log2, z = (tile * kPTile >> p.c.page_log2) + pages;
            if (held >= 0 && held_b == wk.b && held_h == wk.h && a >= held && z <= held + 32) return;
            held = a;
            held_b = wk.b;
            held_h = wk.h;
            const int pg = held + lane;
            page = p.c.pages;  // beyond the cache: the copy reads zeros
            ks = 1.f;
            lvs = 0.f;
            if (((long long)pg << p.c.page_log2) < wk.kv_len) {
                page = p.n.table[(size_t)wk.b * p.n.table_stride + pg];
                if (page < 0 || page >= p.c.pages) {
                    atomicOr(p.err, kDevErrAttnInput);
                    page = p.c.pages;
                } else {
                    ks = p.c.ks[(size_t)page * p.c.heads + wk.h];
                    lvs = log2f(p.c.vs[(size_t)page * p.c.heads + wk.h]);
                }
            }
        };
        auto send = [&](int tile, bool is_v, long long j) {
            if (item >= kSlots) {
                wait(empty + 8 * slot, ph ^ 1u, kDevErrTimeoutEmpty);
                dead = __any_sync(0xffffffffu, dead);
            }
            const int pg0 = (tile * kPTile >> p.c.page_log2) - held;
            if (!is_v) {  // the scales go with K
                const float a = __shfl_sync(0xffffffffu, ks, pg0 + (lane & 7));
                const float c = __shfl_sync(0xffffffffu, lvs, pg0 + (lane & 7));
                float *const to = sscale + (int)(j % kPScaleRing) * 16;
                if (lane < pages) {
                    to[lane] = a;
                    to[8 + lane] = c;
                }
                __syncwarp();
            }
            if (lane == 0 && !dead) mbar_arrive_expect_tx(full + 8 * slot, T::kSlot);
            __syncwarp();
            const int i = lane & (boxes - 1), half = lane / boxes;
            const int pgi = __shfl_sync(0xffffffffu, page, pg0 + i / page_boxes);
            if (half < kHalves && !dead)
                tma_load_4d(smem_u32(ring) + slot * T::kSlot + half * kPTile * 128 + i * box * 128,
                            is_v ? &map_v : &map_k, half * 128, (tile * kPTile + i * box) & (p.c.page - 1), wk.h, pgi,
                            full + 8 * slot, policy);
            if (++slot == kSlots) {
                slot = 0;
                ph ^= 1u;
            }
            if (!dead) ++item;
        };
        for (long long u = u0; u < u1;) {
            if (wk.tile == wk.tiles) wk.next_block(p);
            const int seg = (int)min((long long)(wk.tiles - wk.tile), u1 - u);
            hold(wk.tile, wk.tile);
            send(wk.tile, false, u - u0);
            for (int k = 0; k < seg; ++k) {
                const int tile = wk.tile + k;
                if (k + 1 < seg) {
                    hold(tile, tile + 1);
                    send(tile + 1, false, u - u0 + k + 1);
                }
                send(tile, true, 0);
            }
            u += seg;
            wk.tile += seg;
        }
        // the last copies have landed before the CTA ends
        for (long long i = item > kSlots ? item - kSlots : 0; i < item; ++i)
            if (!mbar_wait_bounded(full + 8 * (int)(i % kSlots), (unsigned)(i / kSlots) & 1u)) {
                if (lane == 0) atomicOr(p.err, kDevErrTimeoutDrain);
                break;
            }
    } else if (warp == kPWarpMma) {
        // ---------------------------------------------------------- MMA issuer
        int slot = 0;
        unsigned ph = 0, seg_ph = 0;
        const uint32_t q0 = smem_u32(sq), r0 = smem_u32(ring);
        auto next_slot = [&]() {
            if (++slot == kSlots) {
                slot = 0;
                ph ^= 1u;
            }
        };
        auto scores = [&](long long j) {  // S(j) = (Qa + Qb) K^T
            wait(full + 8 * slot, ph, kDevErrTimeoutFull);
            tc::fence_after_sync();
            if (lane == 0 && !dead) {
                mbar_arrive(s_full + 8 * (uint32_t)(j & 1));  // hands the page scales on, which came with K
                const uint32_t d = tmem + kPColS + (uint32_t)(j & 1) * kPTile, k0 = r0 + slot * T::kSlot;
#pragma unroll
                for (int half = 0; half < kHalves; ++half)
#pragma unroll
                    for (int s = 0; s < 4; ++s)
#pragma unroll
                        for (int term = 0; term < 2; ++term)
                            mma_f8_ss(d,
                                      tc::smem_desc_sw128(q0 + (term * kHalves + half) * kPRows * 128 + s * 32, 1024),
                                      tc::smem_desc_sw128(k0 + half * kPTile * 128 + s * 32, 1024),
                                      idesc_f8(kPRows, kPTile), half + s + term > 0);
                tc::commit(empty + 8 * slot);
                tc::commit(s_full + 8 * (uint32_t)(j & 1));
            }
            __syncwarp();
            next_slot();
        };
        for (long long u = u0; u < u1;) {
            if (wk.tile == wk.tiles) wk.next_block(p);
            const int seg = (int)min((long long)(wk.tiles - wk.tile), u1 - u);
            wait(q_full, seg_ph, kDevErrTimeoutFull);
            scores(u - u0);
            for (int k = 0; k < seg; ++k) {
                const long long j = u - u0 + k;
                if (k + 1 < seg) scores(j + 1);
                if (k == 0 && u > u0) wait(o_free, seg_ph ^ 1u, kDevErrTimeoutEmpty);  // the last block's output is read
                wait(p_full + 8 * (uint32_t)(j & 1), (unsigned)(j >> 1) & 1u, kDevErrTimeoutFull);
                wait(full + 8 * slot, ph, kDevErrTimeoutFull);
                tc::fence_after_sync();
                if (lane == 0 && !dead) {
                    const uint32_t s = tmem + kPColS + (uint32_t)(j & 1) * kPTile, v0 = r0 + slot * T::kSlot;
#pragma unroll
                    for (int blk = 0; blk < 4; ++blk)
#pragma unroll
                        for (int term = 0; term < 2; ++term)
                            mma_mxf8_ts(tmem, s + blk * 32 + term * 8, smem_desc_mn_sw128(v0 + blk * 32 * 128, kPTile * 128),
                                        idesc_mxf8(kPRows, DP, blk), s + (term ? kPColSfA2 : kPColSfA), s + kPColSfB,
                                        k > 0 || blk + term > 0);
                    tc::commit(empty + 8 * slot);
                    tc::commit(pv_done + 8 * (uint32_t)(j & 1));
                    if (k + 1 == seg) tc::commit(o_full);
                }
                __syncwarp();
                next_slot();
            }
            u += seg;
            wk.tile += seg;
            seg_ph ^= 1u;
        }
    } else if (warp < kPSoftWarps) {
        // ------------------------------------------------------------- softmax
        const int wg = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's lanes of tensor memory
        float qs = 0.f;
        int lim = -1;
        // The block's query rows as two swizzled E4M3 terms, each row scaled by a power of two to a maximum in
        // [2^7, 2^8); a warp takes 16 rows, eight entries a lane.
        auto load_q = [&](const PrmWalk &w) {
            const int rows = w.q_len * p.g, row0 = w.rb * kPRows;
            constexpr int kL = DP / 8;  // lanes of a row
            const int sub = lane / kL, l8 = lane % kL * 8;
#pragma unroll 4
            for (int r = warp * 16 + sub; r < warp * 16 + 16; r += 32 / kL) {
                const bool on = row0 + r < rows && l8 < p.c.d;
                const int i = on ? (row0 + r) / p.g : 0, hq = w.h * p.g + (on ? row0 + r - i * p.g : 0);
                const uint16_t *const src = p.q.p + (w.t0 + i) * p.q.ts + hq * p.q.hs + l8;
                uint32_t v[4] = {0, 0, 0, 0};
                if (on) {
                    if (p.q.vec) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(src);
                        v[0] = x.x;
                        v[1] = x.y;
                        v[2] = x.z;
                        v[3] = x.w;
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = (uint32_t)src[2 * e] | ((uint32_t)src[2 * e + 1] << 16);
                    }
                }
                float x[8], amax = 0.f, zero = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[2 * e] = __uint_as_float(v[e] << 16);
                    x[2 * e + 1] = __uint_as_float(v[e] & 0xFFFF0000u);
                    amax = fmaxf(amax, fmaxf(fabsf(x[2 * e]), fabsf(x[2 * e + 1])));
                    zero += (x[2 * e] - x[2 * e]) + (x[2 * e + 1] - x[2 * e + 1]);  // NaN for an infinity or NaN
                }
#pragma unroll
                for (int s = kL / 2; s > 0; s >>= 1) {
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s, kL));
                    zero += __shfl_xor_sync(0xffffffffu, zero, s, kL);
                }
                const int e = amax > 0.f ? min(max((int)(__float_as_uint(amax) >> 23) - 127 - 7, -119), 119) : 0;
                const float down = pow2i(-e);
                if (l8 == 0) ssum[r] = pow2i(e) * p.scale_log2 + zero;  // a row that is not finite has no scores
                uint32_t a[2], b[2];
#pragma unroll
                for (int z = 0; z < 2; ++z)
                    two_terms<0>(pack_f16(x[4 * z] * down, x[4 * z + 1] * down),
                                 pack_f16(x[4 * z + 2] * down, x[4 * z + 3] * down), a[z], b[z]);
                const int half = l8 >> 7, c = (l8 & 127) >> 4;
                uint8_t *const to = sq + (half * kPRows + r) * 128 + ((c ^ (r & 7)) << 4) + (l8 & 8);
                *reinterpret_cast<uint2 *>(to) = make_uint2(a[0], a[1]);
                *reinterpret_cast<uint2 *>(to + kHalves * kPRows * 128) = make_uint2(b[0], b[1]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        };
        if (wk.tile == wk.tiles) wk.next_block(p);
        load_q(wk);
        bool first_segment = true;
        unsigned seg_ph = 0;
        long long seg_item = 0;  // the ring's item that the segment's K0 is
        for (long long u = u0; u < u1;) {
            const int seg = (int)min((long long)(wk.tiles - wk.tile), u1 - u);
            const int rows = wk.q_len * p.g, row0 = wk.rb * kPRows, start = wk.kv_len - wk.q_len;
            const int all_see = max(0, start + row0 / p.g + 1);
            const int some_see = max(0, start + (min(row0 + kPRows, rows) - 1) / p.g + 1);
            named_barrier(kPBarSoft, kPSoft);  // every row's scale is known
            qs = ssum[row];
            lim = row0 + row < rows ? start + (row0 + row) / p.g : -1;
            if (wg == 0) sref[row] = -INFINITY;
            for (int d = threadIdx.x; d < DP; d += kPSoft) nan_from[d] = 0x7FFFFFFF;
            named_barrier(kPBarSoft, kPSoft);
            float nref = -INFINITY, l = 0.f;
            for (int k = 0; k < seg; ++k) {
                const long long j = u - u0 + k;
                if ((int)(j & 1) != wg) continue;
                const int tile = wk.tile + k, tok_t = tile * kPTile;
                const uint32_t s_col = tmem + kPColS + (uint32_t)wg * kPTile + lanes;
                wait(s_full + 8 * wg, (unsigned)(j >> 1) & 1u, kDevErrTimeoutFull);
                dead = __any_sync(0xffffffffu, dead);
                tc::fence_after_sync();
                const float *const sc = sscale + (int)(j % kPScaleRing) * 16;
                const bool edge = tok_t + kPTile > all_see;
                float E[4];
                float e_max = -INFINITY;
#pragma unroll
                for (int blk = 0; blk < 4; ++blk) {
                    uint32_t v[32];
                    tmem_ld32(s_col + blk * 32, v);
                    const int pa = blk * 32 >> p.c.page_log2, pb = (blk * 32 + 16) >> p.c.page_log2;
                    float f0 = sc[pa] * qs, f1 = sc[pb] * qs;
                    f0 = f0 == 0.f ? 1e-38f : f0;  // not -inf * 0 for a token that is not seen
                    f1 = f1 == 0.f ? 1e-38f : f1;
                    const float lv0 = sc[8 + pa], lv1 = sc[8 + pb];
                    tc::wait_ld();
                    float x[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(v[i]);
                    if (edge) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (tok_t + blk * 32 + i > lim) x[i] = -INFINITY;
                    }
                    float m0 = x[0], m1 = x[16];
#pragma unroll
                    for (int i = 1; i < 16; ++i) {
                        m0 = fmaxf(m0, x[i]);
                        m1 = fmaxf(m1, x[16 + i]);
                    }
                    m0 *= f0;
                    m1 *= f1;
                    const float W = fmaxf(m0 + lv0, m1 + lv1), n = fmaxf(m0, m1);
                    if (n > nref + kPRefSlack) {  // the total's own reference
                        l = nref > -INFINITY ? l * exp2_approx(nref - n) : 0.f;
                        nref = n;
                    }
                    const float e = W > -INFINITY ? ceilf(W) : 0.f;
                    E[blk] = W > -INFINITY ? e : -INFINITY;
                    e_max = fmaxf(e_max, E[blk]);
                    const float c0 = lv0 - e + kWeightLift, c1 = lv1 - e + kWeightLift;
                    const float ref = nref > -INFINITY ? nref : 0.f;
                    const bool apart = fabsf(lv0 - lv1) > 32.f;  // two pages whose weights one exponent does not hold
                    if (apart) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            l += exp2_approx(fmaf(x[i], f0, -ref)) + exp2_approx(fmaf(x[16 + i], f1, -ref));
                    }
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        x[i] = exp2_approx(fmaf(x[i], f0, c0));
                        x[16 + i] = exp2_approx(fmaf(x[16 + i], f1, c1));
                        s0 += x[i];
                        s1 += x[16 + i];
                    }
                    if (!apart) {
                        l = fmaf(s0, exp2_approx(-c0 - ref), l);
                        l = fmaf(s1, exp2_approx(-c1 - ref), l);
                    }
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        two_terms<kPSecond>(pack_f16(x[4 * i], x[4 * i + 1]), pack_f16(x[4 * i + 2], x[4 * i + 3]),
                                            pk[i], pk[8 + i]);
                    tc::st_32x32b_x16(s_col + blk * 32, pk);
                }
                if (edge) {
                    // A zero weight does not hide a NaN: codes that nobody sees become zeros, a NaN that only
                    // some rows see is noted by entry and token (rows see all tokens from one on).
                    const long long iv = seg_item + (k + 1 < seg ? 2 * k + 2 : 2 * k + 1);  // V(k): K0 K1 V0 K2 V1 ...
                    wait(full + 8 * (uint32_t)(iv % kSlots), (unsigned)(iv / kSlots) & 1u, kDevErrTimeoutFull);
                    const int tok = tok_t + row;
                    uint8_t *const vt = ring + (iv % kSlots) * T::kSlot + row * 128;
                    if (tok >= all_see) {
                        for (int c = 0; c < kHalves * 8; ++c) {
                            uint4 *const at4 = reinterpret_cast<uint4 *>(vt + (c >> 3) * kPTile * 128 + ((c ^ row) & 7) * 16);
                            uint4 w4 = tok >= some_see ? make_uint4(0, 0, 0, 0) : *at4;
                            uint32_t *const w = reinterpret_cast<uint32_t *>(&w4);
                            bool changed = tok >= some_see;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t bad = ((w[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                                if (bad) {
                                    changed = true;
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        if (bad >> (8 * e) & 0x80u) {
                                            atomicMin(&nan_from[c * 16 + 4 * i + e], tok);
                                            w[i] &= ~(0xFFu << (8 * e));
                                        }
                                }
                            }
                            if (changed) *at4 = w4;
                        }
                    }
                    fence_proxy_async_smem();
                }
                // ---- scale factors, in the order of the tiles
                if (k > 0) wait(fin + 8 * (wg ^ 1), (unsigned)((j - 1) >> 1) & 1u, kDevErrTimeoutFull);
                float ref = sref[row];
                const bool raise = ref > -INFINITY && e_max > ref + kPRefSlack;
                if (__any_sync(0xffffffffu, raise)) {
                    // O so far is in units of the old reference
                    wait(pv_done + 8 * (wg ^ 1), (unsigned)((j - 1) >> 1) & 1u, kDevErrTimeoutFull);
                    dead = __any_sync(0xffffffffu, dead);
                    tc::fence_after_sync();
                    const float f = raise ? exp2_approx(fmaxf(ref - e_max, -126.f)) : 1.f;
                    for (int c = 0; c < DP; c += 32) {
                        uint32_t v[32];
                        tmem_ld32(tmem + lanes + c, v);
                        tc::wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                        tc::st_32x32b_x32(tmem + lanes + c, v);
                    }
                }
                if (raise || ref == -INFINITY) {
                    ref = e_max;
                    sref[row] = ref;
                }
                const float bias = ref > -INFINITY ? 127.f - ref : 0.f;
                uint32_t sf = 0;
#pragma unroll
                for (int blk = 0; blk < 4; ++blk)
                    sf |= (uint32_t)fminf(fmaxf(E[blk] + bias, 0.f), 254.f) << (8 * blk);
                tmem_st1(s_col + kPColSfA + (warp & 3), sf);
                tmem_st1(s_col + kPColSfA2 + (warp & 3), __vsubus4(sf, 0x01010101u * kPSecond));
                const uint32_t ones[8] = {0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu,
                                          0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu};
                tmem_st8(s_col + kPColSfB, ones);
                tc::wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(fin + 8 * wg);
                    mbar_arrive(p_full + 8 * wg);
                }
            }
            named_barrier(kPBarSoft, kPSoft);  // every tile's weights are made, so every S is done with the queries
            const float my_ref = sref[row];
            ssum[(wg * kPRows + row) * 2] = nref;
            ssum[(wg * kPRows + row) * 2 + 1] = l;
            named_barrier(kPBarSoft, kPSoft);
            float sum, inv, n;
            {
                const float n0 = ssum[2 * row], n1 = ssum[2 * (kPRows + row)];
                n = fmaxf(n0, n1);
                const float r = n > -INFINITY ? n : 0.f;
                sum = exp2_approx(n0 - r) * ssum[2 * row + 1] + exp2_approx(n1 - r) * ssum[2 * (kPRows + row) + 1];
                inv = attn_inverse(n > -INFINITY ? my_ref - n : 0.f, sum);
            }
            named_barrier(kPBarSoft, kPSoft);
            // ---- the next block's queries, so that its first scores are made while this one's output is read
            PrmWalk nx = wk;
            nx.tile += seg;
            if (u + seg < u1) {
                if (nx.tile == nx.tiles) nx.next_block(p);
                load_q(nx);
            }
            // ---- output: half of the columns each
            const bool whole = seg == wk.tiles;
            float *const part = p.partials + ((size_t)blockIdx.x * 2 + (first_segment ? 0 : 1)) * p.slot_floats;
            wait(o_full, seg_ph, kDevErrTimeoutFull);
            dead = __any_sync(0xffffffffu, dead);
            tc::fence_after_sync();
            if (!whole && wg == 0) *reinterpret_cast<float4 *>(part + 4 * row) = make_float4(my_ref, n, sum, 0.f);
            for (int c = wg * (DP / 2); c < (wg + 1) * (DP / 2); c += 32) {
                uint32_t v[32];
                tmem_ld32(tmem + lanes + c, v);
                tc::wait_ld();
                if (some_see > all_see) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (lim >= nan_from[c + i]) v[i] = 0x7FC00000u;
                }
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 x = make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]),
                                                 __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
                    if (whole)
                        attn_store4(p, wk.t0, wk.h, row0 + row, rows, c + i, x, inv);
                    else
                        *reinterpret_cast<float4 *>(part + 4 * kPRows + ((c + i) / 4 * kPRows + row) * 4) = x;
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
            if (!whole) {
                const long long ub = wk.first, ue = wk.first + wk.tiles;
                const int ca = (int)(((ub + 1) * C - 1) / U), cb = (int)((ue * C - 1) / U);
                __threadfence();
                named_barrier(kPBarSoft, kPSoft);
                if (threadIdx.x == 0) {
                    const unsigned old = count_part(p.counters + ca);
                    sh_last = old == (unsigned)(cb - ca);
                    if (sh_last) p.counters[ca] = 0;
                }
                named_barrier(kPBarSoft, kPSoft);
                if (sh_last && row0 + row < rows) {
                    float top = -INFINITY, top_n = -INFINITY;
                    for (int c = ca; c <= cb; ++c) {
                        const float2 x = __ldcg(reinterpret_cast<const float2 *>(attn_part(p, c, ub, U, C) + 4 * row));
                        top = fmaxf(top, x.x);
                        top_n = fmaxf(top_n, x.y);
                    }
                    const bool any = top_n > -INFINITY;
                    float total = 0.f;
                    for (int c = ca; c <= cb; ++c) {
                        const float4 x = __ldcg(reinterpret_cast<const float4 *>(attn_part(p, c, ub, U, C) + 4 * row));
                        total = fmaf(exp2_approx(x.y - (any ? top_n : 0.f)), x.z, total);
                    }
                    const float joined = attn_inverse(any ? top - top_n : 0.f, total);
                    for (int d = wg * (DP / 2); d < (wg + 1) * (DP / 2); d += 4) {
                        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                        for (int c = ca; c <= cb; ++c) {
                            const float *const x = attn_part(p, c, ub, U, C);
                            const float f = exp2_approx(__ldcg(x + 4 * row) - (any ? top : 0.f));
                            const float4 w = __ldcg(reinterpret_cast<const float4 *>(x + 4 * kPRows + (d / 4 * kPRows + row) * 4));
                            v.x = fmaf(f, w.x, v.x);
                            v.y = fmaf(f, w.y, v.y);
                            v.z = fmaf(f, w.z, v.z);
                            v.w = fmaf(f, w.w, v.w);
                        }
                        attn_store4(p, wk.t0, wk.h, row0 + row, rows, d, v, joined);
                    }
                }
            }
            u += seg;
            seg_item += 2 * seg;
            wk = nx;
            seg_ph ^= 1u;
            first_segment = false;
        }
    }
    // ---- every product has been waited for (o_full) by the softmax warps
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kPWarpMma) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kPTmemCols);
    }
}

}  // namespace

constexpr int kPrmStaticSmem = 512;

cudaError_t attn_prompt_set_smem_limit(int smem_optin) {
    if (Prm<256>::kBytes + kPrmStaticSmem > smem_optin || Prm<128>::kBytes + kPrmStaticSmem > smem_optin)
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(attn_prompt_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Prm<128>::kBytes);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(attn_prompt_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Prm<256>::kBytes);
}

cudaError_t launch_attn_prompt(const CUtensorMap &k, const CUtensorMap &v, const AttnParams &p, cudaStream_t stream) {
    if (p.c.d > 128)
        attn_prompt_kernel<256><<<p.ctas, kPThreads, Prm<256>::kBytes, stream>>>(k, v, p);
    else
        attn_prompt_kernel<128><<<p.ctas, kPThreads, Prm<128>::kBytes, stream>>>(k, v, p);
    return cudaGetLastError();
}

}  // namespace nvfp4
