// attn_decode.cu -- attention over the paged 8-bit cache for few query rows:
// single-token decode and the few tokens of a verification step.
//
// For the R = q_len * G query rows that read one kv head (G query heads each)
//
//     y = sum_j p_j V_j / sum_j p_j,   p_j = 2^(s_j - m),
//     s_j = (q . Kcode_j) * qscale * kscale(page) * scale * log2(e),
//
// in one pass over the cache.  The codes go from HBM to shared memory as they
// are stored and become f16 (exactly) in registers on their way into
// mma.sync; 2 bytes are read for 4 R flops, so HBM bounds it.
//
// V's scale.  With w_j = s_j + log2 vscale(page), m the running maximum of w
// and n that of s, the product's weights are 2^(w_j - m + 8) (f16) and the sum
// takes 2^(s_j - n) (fp32): the scales of the pages cost nothing per entry, and
// each weight is rounded relative to what it contributes, whatever the scales
// are.  m and n are left as they are until a weight would exceed 2^15 (f16 ends
// at 2^16), so that most tiles rescale nothing; f16 keeps weights down to 2^-24.
//
// Products.  S^T = K Q^T with 16 tokens as the M rows and 8 query rows as N;
// the order of the head's entries within a k step is free, so that a lane's
// 16-byte load of a token's codes is four k steps of A.  O^T = V^T P^T with 16
// entries of the head as M; P^T comes from S^T's accumulators by an 8x8
// register transpose, and a pair of tokens' codes is interleaved by a byte
// permutation before the conversion.  Both accumulators have the same query
// rows in the same lanes, so the softmax state needs no exchange but the
// maximum over a warp's 16 tokens.
//
// Work split.  A unit is one tile of 64 tokens of one (sequence, kv head); a
// block's (sequence's and head's) own cost counts as kOver units more.  The
// units are numbered in that order and the persistent grid (a CTA an SM) takes
// equal contiguous ranges, whatever the lengths.  A block of several CTAs
// leaves partial results in the workspace, which a second kernel joins in CTA
// order (the result is the same in every run), a CTA for each row; joined by
// the block's last CTA they cost 9 us more for 131071 tokens.
//
// Warps.  Eight consumer warps form two or four teams, which take the CTA's
// tiles in turn, 16 or 32 tokens a warp, with their own softmax state, merged at
// a block's end.  Each team has its own producer warp (or one for K and one for
// V), which feeds the team's stages of the ring by TMA: asking for a tile takes
// about 600 cycles, and HBM delivers one in 700 (64 x 128 of K and V), so that a
// single producer held the kernel at two thirds of HBM's rate.
//
// Measured: 64 sequences of 1 to 4096 tokens, 32 + 8 heads of 128: 404 MB in 71
// us, 5.7 TB/s (0.84 of a plain copy's rate).  131071 tokens of one, 24 + 4
// heads of 256: 269 MB in 51 us, 5.3 TB/s; its main loop runs at 6.6 TB/s, the
// rest are the 3 us until the first tile is asked for, the merge and the join.
#include "attn.cuh"

namespace nvfp4 {

namespace {

constexpr int kTile = 64;                   // tokens of a unit
constexpr int kConsWarps = 8;
constexpr int kCons = kConsWarps * 32;
constexpr int kDecThreads = kCons + 128;    // + the producers' warpgroup
// Registers: 12 warps are launched with 168 each (504 a lane on each of the
// four schedulers); the producers' warpgroup gives up 112 of them and the
// consumers' two take 56 more each: 56 + 2 * 224 = 504.
constexpr int kProdRegs = 56, kConsRegs = 224;
constexpr int kMaxStages = 12;
constexpr int kBarCons = 1;                 // named barrier of the consumer warps
constexpr int kMaxCtas = 160;               // of the grid
constexpr int kAloneBytes = 256 * 1024;     // codes of a block that a CTA reads alone
constexpr float kWeightSlack = 7.f;         // weights are 2^kWeightLift at the maximum and at most 2^7 above
constexpr float kSumSlack = 60.f;

template <int DP, int NT>
struct Dec {
    static constexpr int kHalves = DP / 128;
    static constexpr int kRows = 8 * NT;
    static constexpr int kSub = DP * NT <= 256 ? 2 : 1;       // blocks of 16 tokens that a warp takes together
    static constexpr int kTeam = kTile / (16 * kSub);         // warps of a tile
    static constexpr int kTeams = kConsWarps / kTeam;
    // Tiles' worth of a block's queries and merge.  (6 and 3: 73 us for 64 sequences of up to 4096, 50 us for 16 of
    // up to 8191; these: 71 and 46.)
    static constexpr int kOver = DP == 128 ? 10 : 7;
    static constexpr int kFeeds = 4 / kTeams;                 // producer warps of a team: one, or one for K and one for V
    static constexpr int kStage = 2 * kTile * DP;                             // K then V
    static constexpr int kQ = kRows * DP * 2;                                 // f16 query fragments
    static constexpr int kCols = NT == 1 ? 128 : 64;          // entries of the head that are merged at a time
    static constexpr int kMergeStride = kCols + 4;            // floats: no bank conflicts
    static constexpr int kMerge = kConsWarps * kRows * kMergeStride * 4;
    static constexpr int kMisc = 8 * 2 * kMaxStages + kMaxStages * 8 * 4 + 3 * kConsWarps * kRows * 4 + DP * 4 + 256;
    static constexpr int kFixed = kQ + kMerge + kMisc;
    // A multiple of the teams, so that a stage always belongs to the same one:
    // it then sees every phase of the stage's barrier.  A team that met a stage
    // only every few rounds could take the parity of a round that has not
    // landed for that of the one before it.
    static constexpr int stages(int smem) {
        const int s = (smem - 1024 - kFixed) / kStage;
        return (s < kMaxStages ? s : kMaxStages) / kTeams * kTeams;
    }
    static constexpr int bytes(int stages) { return 1024 + kFixed + stages * kStage; }
};

// Token (row of the tile's 16) of accumulator row r: such that the eight lanes
// of a 16-byte load phase meet eight different bank groups of the swizzled
// tile, for K (rows g, chunks t) and for V (rows 2t, chunks g).
__device__ __forceinline__ int token_of(int r) {
    return (((r ^ (r >> 2)) & 1) << 2) | (r & 2) | ((r >> 2) & 1) | (r & 8);
}

// a / b, a 32-bit division where both fit.
__device__ __forceinline__ long long div_units(long long a, long long b) {
    return (a | b) >> 32 == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// U units over C CTAs: the first `more` take one more than `each`.
struct DecShare {
    long long each, more;
    __device__ DecShare(long long U, long long C) : each(div_units(U, C)), more(U - each * C) {}
    __device__ long long begin(int c) const { return c * each + min((long long)c, more); }
    __device__ int owner(long long u) const {
        const long long head = more * (each + 1);
        return (int)(u < head ? div_units(u, each + 1) : more + div_units(u - head, each));
    }
};

// A block (sequence, kv head) and where this CTA's range stands in it.  A
// block's first `over` units stand for what it costs beside its tiles.
struct DecWalk {
    int b, h, unit;           // next unit of the block
    int t0, q_len, kv_len;
    int tiles;                // of the block
    int over;
    long long first;          // number of the block's first unit
    __device__ static int block_tiles(int kv_len) { return max(1, (kv_len + kTile - 1) / kTile); }
    __device__ void load(const AttnParams &p) {
        kv_sequence(p.n, b, &t0, &q_len, &kv_len);
        tiles = block_tiles(kv_len);
    }
    // The unit `u`, in sequence `seq`, whose first unit is `base`.
    __device__ void begin(const AttnParams &p, int seq, long long base, long long u, int over_units) {
        b = seq;
        over = over_units;
        load(p);
        h = (int)div_units(u - base, tiles + over);
        first = base + (long long)h * (tiles + over);
        unit = (int)(u - first);
    }
    // The range's next tiles (of one block): begin .. end, none at its end.
    __device__ bool next(const AttnParams &p, long long u1, int *begin, int *end) {
        for (;;) {
            if (first + unit >= u1) return false;
            if (unit == tiles + over) {
                first += unit;
                unit = 0;
                if (++h == p.c.heads) {
                    h = 0;
                    do {
                        ++b;
                        load(p);
                    } while (q_len == 0);
                }
            }
            const int from = unit;
            unit = (int)min((long long)(tiles + over), u1 - first);
            *begin = max(0, from - over);
            *end = unit - over;
            if (*end > *begin) return true;
        }
    }
};

// A block of several parts: one record a block where the CTAs suffice for
// that, else one a CTA, for the block that begins in it and that others continue.
struct DecJoin {
    int parts;  // 0: there is none
    int slot;   // of the first part; the others are the following CTAs' first
    int t0, h, rows;
};
__device__ __forceinline__ bool joins_by_block(const AttnParams &p) {
    return (long long)p.n.b * p.c.heads <= p.ctas;
}
static_assert(sizeof(DecJoin) <= kAttnJoinBytes, "a record of the workspace");
__device__ __forceinline__ DecJoin *decode_joins(const AttnParams &p, int cta) {
    return reinterpret_cast<DecJoin *>(reinterpret_cast<uint8_t *>(p.partials + (size_t)p.ctas * 2 * p.slot_floats) +
                                       (size_t)cta * kAttnJoinBytes);
}

// Bits of the bytes of `v` that hold NaN (0x7F or 0xFF): 0x80 in each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t v) { return ((v & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

template <int DP, int NT>
__global__ void __launch_bounds__(kDecThreads, 1)
    attn_decode_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                       const AttnParams p, const int stages, const bool alone) {
    using T = Dec<DP, NT>;
    constexpr int kRows = T::kRows, kHalves = T::kHalves;
    extern __shared__ uint8_t smem_dyn[];
    __shared__ long long sh_scan[kDecThreads / 32], sh_base;
    __shared__ int sh_seq;
    uint8_t *const smem = smem_dyn + ((1024u - (smem_u32(smem_dyn) & 1023u)) & 1023u);
    const uint32_t sring = smem_u32(smem);
    uint8_t *at = smem + stages * T::kStage;
    uint2 *const sq = reinterpret_cast<uint2 *>(at);                 // [DP / 16][NT][32] B fragments
    at += T::kQ;
    float *const merge = reinterpret_cast<float *>(at);              // [warp][row][kMergeStride]
    at += T::kMerge;
    const uint32_t full = smem_u32(at), empty = full + 8 * kMaxStages;
    at += 16 * kMaxStages;
    float *const sscale = reinterpret_cast<float *>(at);             // [stage][2][4]: k scale, log2 of v scale
    at += kMaxStages * 8 * 4;
    float *const wm = reinterpret_cast<float *>(at);                 // [warp][row] maxima of w and s, sums
    float *const wn = wm + kConsWarps * kRows;
    float *const wl = wn + kConsWarps * kRows;
    int *const nan_from = reinterpret_cast<int *>(wl + kConsWarps * kRows);  // [DP] first token whose V is NaN there
    float *const qscale = reinterpret_cast<float *>(nan_from + DP);  // [row]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int B = p.n.b;

    // ---- units of all sequences, and where this CTA's range begins
    if (threadIdx.x < stages) {
        mbar_init(full + 8 * threadIdx.x, T::kFeeds);
        mbar_init(empty + 8 * threadIdx.x, T::kTeam);
        fence_barrier_init();
    }
    griddep_wait();
    if (threadIdx.x == 0) {
        griddep_launch_dependents();  // the joining kernel's CTAs may come as these leave
        if (!joins_by_block(p)) decode_joins(p, blockIdx.x)->parts = 0;
    }
    const int chunk = B <= kDecThreads ? 1 : (B + kDecThreads - 1) / kDecThreads;
    const int b0 = threadIdx.x * chunk, b1 = min(B, b0 + chunk);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
        int t0, q_len, kv_len;
        if (!kv_sequence(p.n, b, &t0, &q_len, &kv_len) && blockIdx.x == 0) atomicOr(p.err, kDevErrAttnInput);
        if (q_len > 0) {
            mine += (long long)(alone ? 1 : DecWalk::block_tiles(kv_len) + T::kOver) * p.c.heads;
        }
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sh_scan[warp] = incl;
    __syncthreads();
    long long U = 0;
    for (int w = 0; w < kDecThreads / 32; ++w) {
        if (w < warp) incl += sh_scan[w];
        U += sh_scan[w];
    }
    const long long C = min((long long)p.ctas, U);
    if (blockIdx.x >= C) return;
    const DecShare share(U, C);
    const long long u0 = share.begin(blockIdx.x);
    long long u1 = share.begin(blockIdx.x + 1);
    if (u0 >= incl - mine && u0 < incl) {
        long long base = incl - mine;
        for (int b = b0; b < b1; ++b) {
            int t0, q_len, kv_len;
            kv_sequence(p.n, b, &t0, &q_len, &kv_len);
            const long long n = q_len > 0 ? (long long)(alone ? 1 : DecWalk::block_tiles(kv_len) + T::kOver) * p.c.heads : 0;
            if (u0 < base + n) {
                sh_seq = b;
                sh_base = base;
                break;
            }
            base += n;
        }
    }
    __syncthreads();
    DecWalk wk;
    if (alone) {  // a unit was a block: from here on the range is these blocks' tiles
        int left = (int)(u1 - u0), h = (int)(u0 - sh_base);
        u1 = 0;
        wk.h = h;
        for (wk.b = sh_seq; left > 0; ++wk.b, h = 0) {
            wk.load(p);
            if (wk.q_len == 0) continue;
            const int n = min(left, p.c.heads - h);
            u1 += (long long)n * wk.tiles;
            left -= n;
        }
        wk.b = sh_seq;
        wk.load(p);
        wk.unit = wk.over = 0;
        wk.first = 0;
    } else {
        wk.begin(p, sh_seq, sh_base, u0, T::kOver);
    }
    bool dead = false;  // a wait gave up: no more waiting, no more copies

    if (warp >= kConsWarps) {
        // ----------------------------------------------------------- producers
        // Four warps: asking for a tile takes one about 600 cycles, and a tile's share of the HBM's time is
        // 700 (D = 128).
        set_max_regs_dec<kProdRegs>();
        constexpr int kFeeds = T::kFeeds;
        const int team = (warp - kConsWarps) / kFeeds, feed = (warp - kConsWarps) % kFeeds;
        const int box = min(p.c.page, kTile), boxes = kTile / box;  // pages of a tile
        const uint64_t policy = l2_policy_evict_first();
        fence_proxy_async_global();
        int st = team;
        unsigned ph = 0;
        int held = -1, held_b = -1, held_h = -1;  // first page number that the lanes hold, 32 in all
        int page = 0;
        float ks = 1.f, lvs = 0.f;
        int sent = 0, ahead = team;  // tiles until this team's next
        int tile, end;
        while (!dead && wk.next(p, u1, &tile, &end)) {
            for (tile += ahead; tile < end; tile += T::kTeams) {
                const int seen = wk.kv_len, h = wk.h;  // slots beyond hold nothing
                const int pg0 = tile * kTile >> p.c.page_log2;
                if (held < 0 || held_b != wk.b || held_h != wk.h || pg0 < held || pg0 + boxes > held + 32) {
                    held = pg0;
                    held_b = wk.b;
                    held_h = wk.h;
                    const int pg = held + lane;
                    page = p.c.pages;  // beyond the cache: the copy reads zeros
                    ks = 1.f;
                    lvs = 0.f;
                    if ((long long)pg << p.c.page_log2 < seen) {
                        page = p.n.table[(size_t)wk.b * p.n.table_stride + pg];
                        if (page < 0 || page >= p.c.pages) {
                            atomicOr(p.err, kDevErrAttnInput);
                            page = p.c.pages;
                        } else {
                            ks = p.c.ks[(size_t)page * p.c.heads + wk.h];
                            lvs = log2f(p.c.vs[(size_t)page * p.c.heads + wk.h]);
                        }
                    }
                }
                int pgs[kTile / 16];
#pragma unroll
                for (int i = 0; i < kTile / 16; ++i) pgs[i] = __shfl_sync(0xffffffffu, page, pg0 - held + (i & (boxes - 1)));
                const int src = pg0 - held + (lane & (boxes - 1));
                const float a = __shfl_sync(0xffffffffu, ks, src), bb = __shfl_sync(0xffffffffu, lvs, src);
                if (sent * T::kTeams >= stages && !mbar_wait_bounded(empty + 8 * st, ph ^ 1u)) {
                    if (lane == 0) atomicOr(p.err, kDevErrTimeoutEmpty);
                    dead = true;
                }
                dead = __any_sync(0xffffffffu, dead);
                if (dead) break;  // no more copies
                ++sent;
                if (feed == 0 && lane < boxes) {
                    sscale[st * 8 + lane] = a;
                    sscale[st * 8 + 4 + lane] = bb;
                }
                __syncwarp();
                if (elect_one()) {
                    const uint32_t bar = full + 8 * st, dst = sring + st * T::kStage;
                    mbar_arrive_expect_tx(bar, T::kStage / kFeeds);
                    const int y = (tile * kTile) & (p.c.page - 1);
#pragma unroll
                    for (int i = 0; i < kTile / 16; ++i) {
                        if (i < boxes) {
#pragma unroll
                            for (int half = 0; half < kHalves; ++half) {
                                const uint32_t to = dst + half * kTile * 128 + i * box * 128;
                                if (kFeeds == 1 || feed == 0)
                                    tma_load_4d(to, &map_k, half * 128, y, h, pgs[i], bar, policy);
                                if (kFeeds == 1 || feed == 1)
                                    tma_load_4d(to + kTile * DP, &map_v, half * 128, y, h, pgs[i], bar, policy);
                            }
                        }
                    }
                }
                __syncwarp();
                if ((st += T::kTeams) >= stages) {
                    st = team;
                    ph ^= 1u;
                }
            }
            ahead = tile - end;
        }
        // the last copies have landed before the CTA ends (its consumers wait for each, unless one gave up)
        const int rounds = stages / T::kTeams;
        for (int i = max(0, sent - rounds); i < sent; ++i)
            if (!mbar_wait_bounded(full + 8 * (team + i % rounds * T::kTeams), (unsigned)(i / rounds) & 1u)) {
                if (lane == 0) atomicOr(p.err, kDevErrTimeoutDrain);
                break;
            }
        return;
    }

    // -------------------------------------------------------------- consumers
    set_max_regs_inc<kConsRegs>();
    constexpr int kSub = T::kSub;
    const int g = lane >> 2, t = lane & 3, team = warp / T::kTeam, first_sub = warp % T::kTeam * kSub;
    const int krow = token_of(g), vrow0 = token_of(2 * t), vrow1 = token_of(2 * t + 1);
    float o[kHalves * 8][NT][4];
    uint2 qf[NT == 1 ? DP / 16 : 1];
    int st = team, ahead = team;
    unsigned ph = 0;
    bool first_segment = true;
    int begin, end;
    while (wk.next(p, u1, &begin, &end)) {
        const int rows = wk.q_len * p.g;
        const int start = wk.kv_len - wk.q_len;
        // ---- the block's query rows as B fragments, each scaled by a power of two to a maximum in [2^7, 2^8)
        for (int r = warp; r < kRows; r += kConsWarps) {
            float x[kHalves * 4];
            float amax = 0.f;
            bool bad = false;  // an infinity or NaN: the row has no scores (and is NaN)
            const bool on = r < rows;
            const int i = on ? p.g_div(r) : 0, hq = wk.h * p.g + (on ? r - i * p.g : 0);
            const uint16_t *src = p.q.p + (wk.t0 + i) * p.q.ts + hq * p.q.hs;
#pragma unroll
            for (int k = 0; k < kHalves * 4; k += 4) {
                const int d = k * 32 + lane * 4;
                uint16_t v[4] = {0, 0, 0, 0};
                if (on && d < p.c.d) {
                    if (p.q.vec) {
                        const uint2 w = *reinterpret_cast<const uint2 *>(src + d);
                        v[0] = (uint16_t)w.x;
                        v[1] = (uint16_t)(w.x >> 16);
                        v[2] = (uint16_t)w.y;
                        v[3] = (uint16_t)(w.y >> 16);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = src[d + e];
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[k + e] = bf16_f32(v[e]);
                    amax = fmaxf(amax, fabsf(x[k + e]));
                    bad |= (v[e] & 0x7F80u) == 0x7F80u;
                }
            }
            bad = __any_sync(0xffffffffu, bad);
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
            const int e = amax > 0.f ? min(max((int)(__float_as_uint(amax) >> 23) - 127 - 7, -119), 119) : 0;
            const float down = pow2i(-e);
            if (lane == 0) qscale[r] = bad ? __int_as_float(0x7FC00000) : pow2i(e) * p.scale_log2;
#pragma unroll
            for (int k = 0; k < kHalves * 4; k += 4) {
                // entries d .. d + 3 = k step (half, it, word), lane t of the fragment, both registers
                const int d = lane * 4, half = k / 4;
                const int it = d >> 6, tt = (d >> 4) & 3, word = (d >> 2) & 3;
                const __half2 lo = __floats2half2_rn(x[k] * down, x[k + 1] * down);
                const __half2 hi = __floats2half2_rn(x[k + 2] * down, x[k + 3] * down);
                sq[(((half * 2 + it) * 4 + word) * NT + (r >> 3)) * 32 + (r & 7) * 4 + tt] =
                    make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
            }
        }
        for (int d = threadIdx.x; d < DP; d += kCons) nan_from[d] = 0x7FFFFFFF;
        named_barrier(kBarCons, kCons);
        if constexpr (NT == 1) {
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) qf[k] = sq[k * 32 + lane];
        }
        float qs[NT][2], m[NT][2], ns[NT][2], l[NT][2];
        int lim[NT][2];  // last token that the row sees
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = 8 * n + 2 * t + c;
                qs[n][c] = qscale[r];
                lim[n][c] = r < rows ? start + p.g_div(r) : -1;
                m[n][c] = ns[n][c] = -INFINITY;
                l[n][c] = 0.f;
            }
        }
#pragma unroll
        for (int k = 0; k < kHalves * 8; ++k)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[k][n][c] = 0.f;
        const int all_see = max(0, start + 1), some_see = wk.kv_len;  // tokens that every, that any row sees

        // ---- the tiles: this warp's tokens of its team's
        int tile = begin + ahead;
        for (; tile < end; tile += T::kTeams) {
            if (!dead && !mbar_wait_bounded(full + 8 * st, ph)) {
                if (lane == 0) atomicOr(p.err, kDevErrTimeoutFull);
                dead = true;
            }
            const uint8_t *const sk = smem + st * T::kStage + first_sub * 16 * 128;
            const uint8_t *const sv = sk + kTile * DP;
            const int base = tile * kTile + first_sub * 16;
            float s[kSub][NT][4];
#pragma unroll
            for (int z = 0; z < kSub; ++z)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[z][n][c] = 0.f;
#pragma unroll
            for (int half = 0; half < kHalves; ++half) {
#pragma unroll
                for (int it = 0; it < 2; ++it) {
                    uint4 v0[kSub], v1[kSub];
#pragma unroll
                    for (int z = 0; z < kSub; ++z) {
                        const uint8_t *const a = sk + half * kTile * 128 + (z * 16 + krow) * 128 +
                                                 (((t + 4 * it) ^ krow) & 7) * 16;
                        v0[z] = *reinterpret_cast<const uint4 *>(a);
                        v1[z] = *reinterpret_cast<const uint4 *>(a + 8 * 128);
                    }
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int ks = (half * 2 + it) * 4 + w;
#pragma unroll
                        for (int z = 0; z < kSub; ++z) {
                            const uint32_t w0[4] = {v0[z].x, v0[z].y, v0[z].z, v0[z].w};
                            const uint32_t w1[4] = {v1[z].x, v1[z].y, v1[z].z, v1[z].w};
                            uint32_t a0, a1, a2, a3;
                            e4m3x4_f16(w0[w], a0, a2);
                            e4m3x4_f16(w1[w], a1, a3);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                const uint2 q = NT == 1 ? qf[NT == 1 ? ks : 0] : sq[(ks * NT + n) * 32 + lane];
                                mma_f16(s[z][n], a0, a1, a2, a3, q.x, q.y);
                            }
                        }
                    }
                }
            }
            // the values' codes, asked for before the softmax
            uint4 v[kSub][4];
            auto load_v = [&](int half) {
#pragma unroll
                for (int z = 0; z < kSub; ++z) {
                    const uint8_t *const a = sv + half * kTile * 128 + z * 16 * 128;
                    v[z][0] = *reinterpret_cast<const uint4 *>(a + vrow0 * 128 + ((g ^ vrow0) & 7) * 16);
                    v[z][1] = *reinterpret_cast<const uint4 *>(a + vrow1 * 128 + ((g ^ vrow1) & 7) * 16);
                    v[z][2] = *reinterpret_cast<const uint4 *>(a + (vrow0 + 8) * 128 + ((g ^ vrow0) & 7) * 16);
                    v[z][3] = *reinterpret_cast<const uint4 *>(a + (vrow1 + 8) * 128 + ((g ^ vrow1) & 7) * 16);
                }
            };
            load_v(0);
            // ---- softmax of the tokens
            const bool edge = base + 16 * kSub > all_see;  // some row does not see some token
            float lvs[kSub];
            bool grow = false;
#pragma unroll
            for (int z = 0; z < kSub; ++z) {
                const int pi = (first_sub + z) * 16 >> p.c.page_log2;  // 0 for pages of a tile or more
                const float ks = sscale[st * 8 + pi];
                lvs[z] = sscale[st * 8 + 4 + pi];
                const int tok0 = base + z * 16 + krow, tok1 = tok0 + 8;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float f = qs[n][c] * ks;
                        s[z][n][c] *= f;
                        s[z][n][2 + c] *= f;
                        if (edge) {
                            if (tok0 > lim[n][c]) s[z][n][c] = -INFINITY;
                            if (tok1 > lim[n][c]) s[z][n][2 + c] = -INFINITY;
                        }
                        const float x = fmaxf(s[z][n][c], s[z][n][2 + c]);
                        grow |= x + lvs[z] > m[n][c] + kWeightSlack || x > ns[n][c] + kSumSlack;
                    }
                }
            }
            if (__any_sync(0xffffffffu, grow)) {  // the rows' maxima over all lanes, only where they matter
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float f[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float y = fmaxf(s[0][n][c], s[0][n][2 + c]), x = y + lvs[0];
#pragma unroll
                        for (int z = 1; z < kSub; ++z) {
                            const float yz = fmaxf(s[z][n][c], s[z][n][2 + c]);
                            y = fmaxf(y, yz);
                            x = fmaxf(x, yz + lvs[z]);
                        }
#pragma unroll
                        for (int o2 = 4; o2 < 32; o2 *= 2) {
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o2));
                            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o2));
                        }
                        x = fmaxf(m[n][c], x);
                        y = fmaxf(ns[n][c], y);
                        f[c] = 1.f;
                        if (y > -INFINITY) {
                            f[c] = exp2_approx(m[n][c] - x);
                            l[n][c] *= exp2_approx(ns[n][c] - y);
                        }
                        m[n][c] = x;
                        ns[n][c] = y;
                    }
#pragma unroll
                    for (int k2 = 0; k2 < kHalves * 8; ++k2) {
                        o[k2][n][0] *= f[0];
                        o[k2][n][1] *= f[1];
                        o[k2][n][2] *= f[0];
                        o[k2][n][3] *= f[1];
                    }
                }
            }
            uint32_t pf[kSub][NT][2];
#pragma unroll
            for (int z = 0; z < kSub; ++z) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float e[4];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const bool any = ns[n][c] > -INFINITY;  // else every weight is 0, or NaN
                        const float ref = any ? m[n][c] - lvs[z] - kWeightLift : 0.f, ref_l = any ? ns[n][c] : 0.f;
                        e[c] = exp2_approx(s[z][n][c] - ref);
                        e[2 + c] = exp2_approx(s[z][n][2 + c] - ref);
                        l[n][c] += exp2_approx(s[z][n][c] - ref_l) + exp2_approx(s[z][n][2 + c] - ref_l);
                    }
                    const __half2 x = __floats2half2_rn(e[0], e[1]), y = __floats2half2_rn(e[2], e[3]);
                    pf[z][n][0] = transpose8x8(*reinterpret_cast<const uint32_t *>(&x));
                    pf[z][n][1] = transpose8x8(*reinterpret_cast<const uint32_t *>(&y));
                }
            }
            // ---- values
#pragma unroll
            for (int half = 0; half < kHalves; ++half) {
                if (half > 0) load_v(half);
                if (edge) {
                    // A zero weight does not hide a NaN: codes that nobody sees become zeros, a NaN that
                    // only some rows see is noted by entry and token (rows see all tokens from one on).
#pragma unroll
                    for (int i = 0; i < 4 * kSub; ++i) {
                        const int tok = base + (i >> 2) * 16 + ((i & 1) ? vrow1 : vrow0) + (i >> 1 & 1) * 8;
                        uint32_t *const w = reinterpret_cast<uint32_t *>(&v[i >> 2][i & 3]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (tok >= some_see) w[j] = 0;
                            const uint32_t bad = nan_bytes(w[j]);
                            if (bad && tok >= all_see) {
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (bad >> (8 * e) & 0x80u) {
                                        atomicMin(&nan_from[half * 128 + 16 * g + 4 * j + e], tok);
                                        w[j] &= ~(0xFFu << (8 * e));
                                    }
                            }
                        }
                    }
                }
#pragma unroll
                for (int z = 0; z < kSub; ++z) {
                    const uint32_t va[4] = {v[z][0].x, v[z][0].y, v[z][0].z, v[z][0].w};
                    const uint32_t vb[4] = {v[z][1].x, v[z][1].y, v[z][1].z, v[z][1].w};
                    const uint32_t vc[4] = {v[z][2].x, v[z][2].y, v[z][2].z, v[z][2].w};
                    const uint32_t vd[4] = {v[z][3].x, v[z][3].y, v[z][3].z, v[z][3].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint32_t sel = y ? 0x7362u : 0x5140u;
                            uint32_t a0, a1, a2, a3;
                            e4m3x4_f16(__byte_perm(va[j], vb[j], sel), a0, a1);
                            e4m3x4_f16(__byte_perm(vc[j], vd[j], sel), a2, a3);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma_f16(o[half * 8 + 2 * j + y][n], a0, a1, a2, a3, pf[z][n][0], pf[z][n][1]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * st);
            if ((st += T::kTeams) >= stages) {
                st = team;
                ph ^= 1u;
            }
        }
        ahead = tile - end;

        // ---- merge of the eight warps, kCols entries of the head at a time
        constexpr int kCols = T::kCols, kStride = T::kMergeStride, kQuads = kCols / 4;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float x = l[n][c];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                if (g == 0) {
                    wm[warp * kRows + 8 * n + 2 * t + c] = m[n][c];
                    wn[warp * kRows + 8 * n + 2 * t + c] = ns[n][c];
                    wl[warp * kRows + 8 * n + 2 * t + c] = x;
                }
            }
        const bool whole = begin == 0 && end == wk.tiles;
        // a part: of the CTA's first block, or of its last, which others continue
        const bool kept = !whole && nvfp4_in_bounds((int)blockIdx.x < p.ctas && rows <= kRows &&
                                                        (first_segment || end < wk.tiles) &&
                                                        4 * kRows + kRows * DP <= p.slot_floats,
                                                    p.err);
        float *const part = p.partials + ((size_t)blockIdx.x * 2 + (first_segment ? 0 : 1)) * p.slot_floats;
        constexpr int kPer = kRows * kQuads / kCons;  // rows of a thread
        const int q4 = threadIdx.x % kQuads;          // its four entries
        float fw[kPer][kConsWarps], inv[kPer];
#pragma unroll 1
        for (int jp = 0; jp < DP / kCols; ++jp) {
            const int half = jp * kCols / 128, j0 = jp * kCols % 128 / 32;
#pragma unroll
            for (int at_jp = 0; at_jp < DP / kCols; ++at_jp)
                if (at_jp == jp) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int y = 0; y < kCols / 32; ++y) {
                                const int k2 = at_jp * (kCols / 16) + 2 * y;
                                *reinterpret_cast<float4 *>(merge + (warp * kRows + 8 * n + 2 * t + c) * kStride + y * 32 +
                                                            g * 4) =
                                    make_float4(o[k2][n][c], o[k2][n][2 + c], o[k2 + 1][n][c], o[k2 + 1][n][2 + c]);
                            }
                }
            named_barrier(kBarCons, kCons);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int r = threadIdx.x / kQuads + i * (kCons / kQuads);
                if (jp == 0) {
                    float top = -INFINITY, top_n = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kConsWarps; ++w) {
                        top = fmaxf(top, wm[w * kRows + r]);
                        top_n = fmaxf(top_n, wn[w * kRows + r]);
                    }
                    const bool any = top_n > -INFINITY;
                    float sum = 0.f;
#pragma unroll
                    for (int w = 0; w < kConsWarps; ++w) {
                        fw[i][w] = exp2_approx(wm[w * kRows + r] - (any ? top : 0.f));
                        sum = fmaf(exp2_approx(wn[w * kRows + r] - (any ? top_n : 0.f)), wl[w * kRows + r], sum);
                    }
                    inv[i] = attn_inverse(any ? top - top_n : 0.f, sum);
                    if (kept && q4 == 0)
                        *reinterpret_cast<float4 *>(part + 4 * r) = make_float4(top, top_n, sum, 0.f);
                }
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kConsWarps; ++w) {
                    const float4 x = *reinterpret_cast<const float4 *>(merge + (w * kRows + r) * kStride + q4 * 4);
                    v.x = fmaf(fw[i][w], x.x, v.x);
                    v.y = fmaf(fw[i][w], x.y, v.y);
                    v.z = fmaf(fw[i][w], x.z, v.z);
                    v.w = fmaf(fw[i][w], x.w, v.w);
                }
                const int d = half * 128 + 16 * (q4 & 7) + 4 * (j0 + (q4 >> 3));
                if (some_see > all_see) {  // entries that are NaN from some token on
                    const int li = r < rows ? start + p.g_div(r) : -1;
                    if (li >= nan_from[d]) v.x = __int_as_float(0x7FC00000);
                    if (li >= nan_from[d + 1]) v.y = __int_as_float(0x7FC00000);
                    if (li >= nan_from[d + 2]) v.z = __int_as_float(0x7FC00000);
                    if (li >= nan_from[d + 3]) v.w = __int_as_float(0x7FC00000);
                }
                if (whole)
                    attn_store4(p, wk.t0, wk.h, r, rows, d, v, inv[i]);
                else if (kept && r < rows)
                    *reinterpret_cast<float4 *>(part + 4 * kRows + r * DP + d) = v;
            }
            named_barrier(kBarCons, kCons);
        }
        const bool by_block = joins_by_block(p);
        const int record = by_block ? wk.b * p.c.heads + wk.h : (int)blockIdx.x;
        if (threadIdx.x == 0 && !alone && begin == 0 && (by_block || !whole) &&
            nvfp4_in_bounds(record >= 0 && record < p.ctas, p.err))
            *decode_joins(p, record) =
                DecJoin{whole ? 0 : share.owner(wk.first + wk.over + wk.tiles - 1) - (int)blockIdx.x + 1,
                        (int)blockIdx.x * 2 + (first_segment ? 0 : 1), wk.t0, wk.h, rows};
        first_segment = false;
    }
}

// Joins the parts of row blockIdx.y of the block of record blockIdx.x.  Groups
// of DP / 4 threads each sum some of the parts, eight of them asked for at
// once; the groups' sums are added in order.
constexpr int kJoinThreads = 512;
template <int DP>
__global__ void __launch_bounds__(kJoinThreads, 2) attn_decode_join_kernel(const AttnParams p, const int block_rows) {
    constexpr int kItems = DP / 4, kGroups = kJoinThreads / kItems, kBatch = 8;
    __shared__ float fac[kMaxCtas], sh_inv;
    __shared__ float4 sums[kGroups][kItems];
    griddep_wait();
    if (joins_by_block(p)) {  // a sequence that brings no tokens has no records
        int t0, q_len, kv_len;
        kv_sequence(p.n, blockIdx.x / p.c.heads, &t0, &q_len, &kv_len);
        if (q_len == 0) return;
    }
    const DecJoin at = *decode_joins(p, blockIdx.x);
    const int r = blockIdx.y;
    if (at.parts == 0 || r >= at.rows) return;
    if (!nvfp4_in_bounds((int)blockIdx.x < p.ctas && at.slot >= 0 && at.parts > 1 && at.parts <= kMaxCtas &&
                             (at.slot >> 1) + at.parts <= p.ctas && at.rows <= block_rows,
                         p.err))
        return;
    const float *const first = p.partials + (size_t)at.slot * p.slot_floats;
    const float *const others = p.partials + (size_t)(at.slot >> 1) * 2 * p.slot_floats;
    auto part_of = [&](int c) { return c == 0 ? first : others + (size_t)c * 2 * p.slot_floats; };
    const int item = threadIdx.x % kItems, group = threadIdx.x / kItems;
    float4 w[kBatch];
    auto load_parts = [&](int c0) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int c = c0 + k * kGroups;
            w[k] = c < at.parts ? __ldcg(reinterpret_cast<const float4 *>(part_of(c) + 4 * block_rows + r * DP + item * 4))
                                : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    load_parts(group);
    if (threadIdx.x < 32) {  // 2^(a part's maximum - all parts'), and the weights' total
        const int lane = threadIdx.x;
        float top = -INFINITY, top_n = -INFINITY, sum = 0.f;
        float4 x[kMaxCtas / 32];
#pragma unroll
        for (int k = 0; k < kMaxCtas / 32; ++k) {
            const int c = lane + 32 * k;
            x[k] = c < at.parts ? __ldcg(reinterpret_cast<const float4 *>(part_of(c) + 4 * r))
                                : make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
            top = fmaxf(top, x[k].x);
            top_n = fmaxf(top_n, x[k].y);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            top_n = fmaxf(top_n, __shfl_xor_sync(0xffffffffu, top_n, o));
        }
        const bool any = top_n > -INFINITY;
#pragma unroll
        for (int k = 0; k < kMaxCtas / 32; ++k) {
            fac[lane + 32 * k] = exp2_approx(x[k].x - (any ? top : 0.f));
            sum = fmaf(exp2_approx(x[k].y - (any ? top_n : 0.f)), x[k].z, sum);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) sh_inv = attn_inverse(any ? top - top_n : 0.f, sum);
    }
    __syncthreads();
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = group; c0 < at.parts; c0 += kBatch * kGroups) {
        if (c0 != group) load_parts(c0);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int c = c0 + k * kGroups;
            if (c < at.parts) {
                v.x = fmaf(fac[c], w[k].x, v.x);
                v.y = fmaf(fac[c], w[k].y, v.y);
                v.z = fmaf(fac[c], w[k].z, v.z);
                v.w = fmaf(fac[c], w[k].w, v.w);
            }
        }
    }
    sums[group][item] = v;
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int i = 1; i < kGroups; ++i) {
        const float4 x = sums[i][item];
        v.x += x.x;
        v.y += x.y;
        v.z += x.z;
        v.w += x.w;
    }
    attn_store4(p, at.t0, at.h, r, at.rows, item * 4, v, sh_inv);
}

template <int DP, int NT>
cudaError_t dec_launch(const CUtensorMap &k, const CUtensorMap &v, const AttnParams &call, int smem,
                       cudaStream_t stream) {
    const int stages = Dec<DP, NT>::stages(smem);
    AttnParams p = call;
    if (p.ctas > kMaxCtas) p.ctas = kMaxCtas;
    // Whole blocks to a CTA, and no second kernel: short ones, if few enough for a CTA each (a sequence of 512 tokens,
    // 32 + 8 heads of 128: 6.1 us so and 8.3 in parts; of 1024 tokens 8.0 and 8.5; of 2048 11.6 and 9.1), or if their
    // tiles cost less than what comes with a block and they fill the CTAs' rounds to two thirds (67 sequences of 34
    // tokens, 32 + 8 heads of 128: 17 us and 19).
    const long long blocks = (long long)p.n.b * p.c.heads, rounds = (blocks + p.ctas - 1) / p.ctas;
    const bool alone = rounds <= 1 ? p.n.max_kv <= kAloneBytes / (2 * DP)
                                   : p.n.max_kv <= Dec<DP, NT>::kOver * kTile && rounds * p.ctas <= blocks + blocks / 2;
    cudaError_t e = launch_behind(attn_decode_kernel<DP, NT>, dim3((unsigned)p.ctas), kDecThreads,
                                  Dec<DP, NT>::bytes(stages), stream, k, v, p, stages, alone);
    if (e != cudaSuccess || alone) return e;
    return launch_behind(attn_decode_join_kernel<DP>,
                         dim3((unsigned)(blocks <= p.ctas ? blocks : p.ctas), (unsigned)(p.n.max_q * p.g)), kJoinThreads, 0,
                         stream, p, (int)Dec<DP, NT>::kRows);
}
template <int DP, int NT>
cudaError_t dec_limit(int smem) {
    return cudaFuncSetAttribute(attn_decode_kernel<DP, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Dec<DP, NT>::bytes(Dec<DP, NT>::stages(smem)));
}

}  // namespace

// The static shared memory of the kernel counts too.
constexpr int kDecStaticSmem = 256;

cudaError_t attn_decode_set_smem_limit(int smem_optin) {
    const int smem = smem_optin - kDecStaticSmem;
    cudaError_t e;
    if ((e = dec_limit<128, 1>(smem)) != cudaSuccess || (e = dec_limit<128, 2>(smem)) != cudaSuccess ||
        (e = dec_limit<256, 1>(smem)) != cudaSuccess)
        return e;
    return dec_limit<256, 2>(smem);
}

cudaError_t launch_attn_decode(const CUtensorMap &k, const CUtensorMap &v, const AttnParams &p, int smem_optin,
                               cudaStream_t stream) {
    const int smem = smem_optin - kDecStaticSmem;
    const bool eight = p.n.max_q * p.g <= 8;  // rows
    if (p.c.d > 128)
        return eight ? dec_launch<256, 1>(k, v, p, smem, stream) : dec_launch<256, 2>(k, v, p, smem, stream);
    return eight ? dec_launch<128, 1>(k, v, p, smem, stream) : dec_launch<128, 2>(k, v, p, smem, stream);
}

}  // namespace nvfp4
