// attn_shared.cu -- attention for a batch whose sequences share long prefixes:
// what is shared, how the work is cut, and the join of its parts.
//
// A row's softmax over all its tokens is the join of softmaxes over any parts of
// them: with (O, m, n, l) a part's weighted sum of values in units of 2^m and
// its weights' total in units of 2^n,
//
//     result = sum_i 2^(m_i - M) O_i / sum_i 2^(n_i - N) l_i  *  2^(M - N),   M = max m_i, N = max n_i.
//
// So a group's rows, neighbours in the batch, are multiplied with the group's
// prefix as those of one sequence that sees all of it (128 rows at a time, by the
// prompt kernel), and each sequence's with its own tokens, in chunks; one kernel
// joins what they leave.  Neither pass fills the GPU by itself: what a CTA of the
// first spends on queries, first tile and output is worth eight of its tiles, and
// the second is bound by latencies too, or by the memory's rate.  They run beside
// each other, the first on as many SMs as its share of the work.
//
// 64 sequences of 510 to 1021 tokens behind 16384, 32 + 8 heads of 128, in a CUDA
// graph: 57 us (135 MB, 20 us at the copy's rate; sequence by sequence 214 us).  The
// plan takes 5.6 us, the pass over the prefix runs from 7 to 43 (on 80 SMs: a tile of
// 128 x 128 takes 1.1 us, most of it softmax), the last chunk ends at 48 and the join at
// 55.  6 groups of 8 behind 7000, 24 + 4 heads of 256: 51 us (18 at the copy's rate; 89).
//
// Where a figure here or in the entry point is "over 14 cases", it is the geometric mean of their times in a CUDA graph,
// three sets of inputs in turn: groups, sequences of all, tokens of each, prefix, most own tokens (us sequence by
// sequence, and by this call):
//   heads of 128, 32 + 8:  1, 64 x 1 over 16384 + 1021 (214, 56);  1, 16 x 1 over 4096 + 2000 (31, 29);  1, 32 x 1 over
//     32768 + 200 (201, 40);  4, 64 x 1 over 4096 + 500 (63, 40);  1, 128 x 1 over 8192 + 700 (229, 72);  1, 8 x 1 over
//     8192 + 300 (23, 23);  1, 4 x 1 over 32768 + 300 (34, 35)
//   heads of 128, 40 + 8:  1, 32 x 5 over 32768 + 300 (339, 147)
//   heads of 256, 24 + 4, gated:  1, 16 x 1 over 8192 + 509 (43, 31);  6, 48 x 1 over 7000 + 700 (89, 51);  1, 64 x 1 over
//     2048 + 200 (53, 31);  2, 8 x 1 over 16384 + 300 (40, 38);  1, 24 x 4 over 8192 + 600 (115, 53);  1, 4 x 1 over
//     8192 + 300 (21, 21)
//
// What is shared of a prefix is what every token of the group sees, whole pages
// and whole tiles of 128 tokens of it: so it needs no masks, and what is left of
// it is read with each sequence's own tokens.
#include "attn.cuh"
#include "attn_units.h"
#include "scan.cuh"

namespace nvfp4 {

namespace {

constexpr int kPlanThreads = 1024;  // at most
constexpr int kLeastStep = 16;      // tokens that chunks are whole multiples of if each has a warp (else kChunkUnit)
constexpr int kPlanTries = 5;       // chunk lengths that are tried (over 14 cases 41.6 us; 3: 42.8, 8: 41.8)
constexpr float kChunkOver = 80.f;  // what a chunk costs besides its tokens, in tokens
constexpr int kPlanHeld = 1024;     // sequences whose lengths the plan keeps in shared memory
// One CTA: the records of groups and sequences.  What it reads is asked for at
// once; the rest is a few barriers, and code that runs once: most of its time goes
// to fetching instructions, so that loops stay loops and numbers in 32 bits (5 to
// 6 us for 16 or 64 sequences).
__global__ void __launch_bounds__(kPlanThreads) attn_shared_plan_kernel(const SharedPlan p) {
    constexpr int kG = kSharedMaxGroups;
    extern __shared__ int plan_smem[];
    __shared__ int warps[2][32];
    __shared__ unsigned long long sh_steps, sh_rows;
    __shared__ int sh_units, sh_tiles, sh_ctas, sh_blocks, sh_items[kPlanTries];
    // by group: first sequence; tokens that all see, then those that are shared; first sequence that holds some; such
    // sequences, then CTAs of a block; first row and rows; the prefix's length, then the first unit of the prompt kernel's
    int *const cu = plan_smem, *const start = cu + kG + 1, *const first = start + kG, *const active = first + kG,
        *const row0 = active + kG, *const tokens = row0 + kG, *const length = tokens + kG;
    // by sequence, for the first kPlanHeld: first row, rows, tokens (then those behind the prefix), group
    int *const s_t0 = length + kG, *const s_q = s_t0 + kPlanHeld, *const s_kv = s_q + kPlanHeld,
        *const s_group = s_kv + kPlanHeld;
    const int G = p.groups, B = p.n.b, unit = max(kPTile, 1 << p.page_log2), T = blockDim.x;
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();  // the prompt kernel's barriers and tensor memory meanwhile
    bool ok = true, neighbours = true, bad = false;  // neighbours: every row belongs to one sequence
#pragma unroll 1
    for (int g = threadIdx.x; g <= G; g += T) {
        const int c = p.group_cu[g], next = g < G ? p.group_cu[g + 1] : B, n = g < G ? p.prefix_lens[g] : 0;
        ok = ok && c >= 0 && next >= c;
        bad = bad || n < 0 || n > p.n.max_kv;
        cu[g] = c;
        if (g < G) {
            length[g] = n < 0 || n > p.n.max_kv ? 0 : n;
            start[g] = first[g] = kMost;
            active[g] = 0;
        }
    }
#pragma unroll 1
    for (int b = threadIdx.x; b < B; b += T) {
        int t0, q_len, kv_len;
        bad = !kv_sequence(p.n, b, &t0, &q_len, &kv_len) || bad;
        neighbours = neighbours && p.n.cu[b + 1] - p.n.cu[b] == q_len && (q_len == 0 || p.n.cu[b] == t0);
        if (b < kPlanHeld) {
            s_t0[b] = t0;
            s_q[b] = q_len;
            s_kv[b] = kv_len;
        }
    }
    if (threadIdx.x < kPlanTries) sh_items[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
        sh_steps = sh_rows = 0;
        sh_units = sh_tiles = sh_ctas = sh_blocks = 0;
    }
    ok = __syncthreads_and(ok);
    neighbours = __syncthreads_and(neighbours);
    if (bad || !ok) atomicOr(p.err, kDevErrAttnInput);
    // (what is nobody's group is behind no prefix; of groups that begin at one sequence all but the last are empty)
    auto sequence = [&](int b, int *t0, int *q_len, int *kv_len, int *group) {
        if (b < kPlanHeld) {
            *t0 = s_t0[b];
            *q_len = s_q[b];
            *kv_len = s_kv[b];
        } else {
            kv_sequence(p.n, b, t0, q_len, kv_len);
        }
        *group = !ok || *kv_len == 0 || b < cu[0] || b >= cu[G] ? -1 : last_at(cu, G, b);
    };
    // ---- what all tokens of a group see
#pragma unroll 1
    for (int b = threadIdx.x; b < B; b += T) {
        int t0, q_len, kv_len, g;
        sequence(b, &t0, &q_len, &kv_len, &g);
        if (g >= 0 && q_len > 0) {  // others see nothing of the prefix
            atomicMin(&start[g], max(0, kv_len - q_len));
            atomicMin(&first[g], b);
            atomicAdd(&active[g], 1);
        }
    }
    __syncthreads();
    auto row_blocks = [&](int q_len) { return (q_len * p.g + p.rows_chunk - 1) >> (p.rows_chunk == 8 ? 3 : 4); };  // a chunk's
    auto blocks_of = [&](int q_len) { return (q_len * p.g + kPRows - 1) / kPRows * p.heads; };  // the prompt kernel's
    auto tiles_of = [&](int kv_len) { return kv_len / kPTile; };
#pragma unroll 1
    for (int g = threadIdx.x; g < G; g += T) {
        int shared = 0, from = 0, rows = 0;
        if (ok && neighbours && active[g] > 1) {
            from = p.n.cu[cu[g]];
            rows = p.n.cu[cu[g + 1]] - from;
            shared = rows > p.max_group_tokens ? 0 : min(length[g], start[g]) & -unit;
        }
        start[g] = shared;
        row0[g] = shared > 0 ? from : 0;
        tokens[g] = shared > 0 ? rows : 0;
        if (shared > 0) {
            atomicAdd(&sh_units, blocks_of(rows) * (tiles_of(shared) + kPOverShared));
            atomicAdd(&sh_tiles, blocks_of(rows) * tiles_of(shared));
        }
    }
    __syncthreads();
    auto own = [&](int b, int *t0, int *q_len, int *kv_len, int *group) {  // what sequence b holds behind its prefix
        sequence(b, t0, q_len, kv_len, group);
        const int shared = *group >= 0 ? start[*group] : 0;
        *kv_len -= shared;
        if (shared == 0) *group = -1;
    };
    // ---- all blocks of rows times their own tokens, and all rows: how long a chunk is
    unsigned long long steps_here = 0, rows_here = 0;
#pragma unroll 1
    for (int b = threadIdx.x; b < B; b += T) {
        int t0, q_len, kv_len, group;
        own(b, &t0, &q_len, &kv_len, &group);
        if (b < kPlanHeld) {
            s_kv[b] = kv_len;
            s_group[b] = group;
        }
        steps_here += (unsigned long long)row_blocks(q_len) * kv_len;
        rows_here += (unsigned long long)(q_len * p.g) * kv_len;
    }
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) {
        steps_here += __shfl_xor_sync(0xffffffffu, steps_here, o);
        rows_here += __shfl_xor_sync(0xffffffffu, rows_here, o);
    }
    if ((threadIdx.x & 31) == 0) {
        atomicAdd(&sh_steps, steps_here);
        atomicAdd(&sh_rows, rows_here);
    }
    __syncthreads();
    auto known = [&](int b, int *t0, int *q_len, int *kv_len, int *group) {  // the same from here on
        if (b < kPlanHeld) {
            *t0 = s_t0[b];
            *q_len = s_q[b];
            *kv_len = s_kv[b];
            *group = s_group[b];
        } else {
            own(b, t0, q_len, kv_len, group);
        }
    };
    const int U = sh_units;
    const float steps = (float)sh_steps * p.heads;
    // (divisions that need not be exact are quick ones: one after the other, they are a part of the kernel's time)
    const float least = fmaxf(fmaxf((float)sh_steps * p.of_steps, (float)U * p.of_units), (float)sh_rows * p.of_rows);
    int chunk = shared_chunk(least);
    // The prompt kernel's CTAs: a unit of it costs as much as unit_steps steps of 16 tokens, a chunk five steps more.
    const float work = steps * 0.0625f + 5.f * __fdividef(steps, (float)chunk), cost = (float)U * p.unit_steps;
    const int share = (int)(p.ctas * __fdividef(cost, fmaxf(cost + work, 1.f)) + 0.5f);
    int C = min(U, max(1, work > 0.f ? min(share, p.ctas - 1) : p.ctas));
    // A block of rows to whole CTAs of its own, each an equal share of its tiles, if that takes hardly more CTAs; else C
    // CTAs share all units, and some have the end of one block and the begin of another (always so: 42.2 us over 14
    // cases from 41.6).
    const int each = C > 0 ? (sh_tiles + C - 1) / C : 1;  // tiles of a CTA
#pragma unroll 1
    for (int g = threadIdx.x; g < G; g += T)
        if (tokens[g] > 0) {
            active[g] = (tiles_of(start[g]) + each - 1) / each;
            atomicAdd(&sh_ctas, blocks_of(tokens[g]) * active[g]);
        }
    // If all chunks can be taken at once, by a warp each: the shortest such length of a few, from that on which would do
    // with nothing left over, unless chunks in turns take less (over 14 cases 41.6 us, always in turns 43.1).
    float takers = fmaxf(1.f, (float)(p.ctas - C) * p.chunk_warps);
    const int shortest = (int)fminf(fmaxf(fmaxf(__fdividef(steps, takers), (float)sh_rows * p.of_rows), 1.f), 1e8f);
    auto length_of = [&](int i) { return (shortest + shortest * i / (kPlanTries - 1) + kLeastStep - 1) & -kLeastStep; };
    int count[kPlanTries] = {}, blocks_here = 0;
    float of_one[kPlanTries];  // (what is off by a last bit only chooses another length)
#pragma unroll
    for (int i = 0; i < kPlanTries; ++i) of_one[i] = __fdividef(1.f, (float)length_of(i));
#pragma unroll 1
    for (int b = threadIdx.x; b < B; b += T) {
        int t0, q_len, kv_len, group;
        known(b, &t0, &q_len, &kv_len, &group);
        const int blocks = kv_len > 0 ? row_blocks(q_len) : 0;
        blocks_here += blocks;
#pragma unroll
        for (int i = 0; i < kPlanTries; ++i) count[i] += blocks * (int)ceilf((float)kv_len * of_one[i]);
    }
#pragma unroll
    for (int i = 0; i < kPlanTries; ++i) {
        count[i] = __reduce_add_sync(0xffffffffu, count[i]);
        if ((threadIdx.x & 31) == 0) atomicAdd(&sh_items[i], count[i]);
    }
    blocks_here = __reduce_add_sync(0xffffffffu, blocks_here);
    if ((threadIdx.x & 31) == 0) atomicAdd(&sh_blocks, blocks_here);
    __syncthreads();
    const bool whole = sh_ctas <= min(work > 0.f ? p.ctas - 1 : p.ctas, C + C / 16);
    if (whole) C = sh_ctas;
    takers = fmaxf(1.f, (float)(p.ctas - C) * p.chunk_warps);
    const float in_turns = __fdividef((__fdividef(steps, (float)chunk) + 0.5f * sh_blocks * p.heads) * kChunkOver + steps, takers) +
                           0.25f * (kChunkOver + chunk);
#pragma unroll 1
    for (int i = 0; i < kPlanTries; ++i)
        if ((float)sh_items[i] * p.heads <= takers) {
            if (kChunkOver + length_of(i) < in_turns) chunk = length_of(i);
            break;
        }
    // ---- where each one's units, chunks and parts begin
    int items = 0, parts = 0, units = 0;  // parts: rows of them
#pragma unroll 1
    for (int g0 = 0; g0 < G; g0 += T) {
        const int g = g0 + threadIdx.x;
        int x[1] = {0}, total[1];
        SharedSeq to = {};
        if (g < G && tokens[g] > 0) {
            to.split = whole ? active[g] : 0;
            x[0] = blocks_of(tokens[g]) * (whole ? to.split : tiles_of(start[g]) + kPOverShared);
        }
        block_sums(x, total, warps);
        if (g < G) {
            to.t0 = row0[g];
            to.q_len = tokens[g];
            to.kv_len = start[g];
            to.row = tokens[g] > 0 ? first[g] : 0;
            to.units = length[g] = units + x[0];
            p.prefixes[g] = to;
        }
        units += total[0];
    }
#pragma unroll 1
    for (int b0 = 0; b0 < B; b0 += T) {
        const int b = b0 + threadIdx.x;
        int t0 = 0, q_len = 0, kv_len = 0, group = -1, chunks = 0, x[2] = {0, 0}, total[2];
        if (b < B) {
            known(b, &t0, &q_len, &kv_len, &group);
            chunks = q_len > 0 ? (kv_len + chunk - 1) / chunk : 0;
            const long long rows = (long long)chunks * q_len * p.g * p.heads;
            x[0] = (int)min((long long)chunks * row_blocks(q_len) * p.heads, (long long)kMost);
            x[1] = (int)min(rows, (long long)kMost);
        }
        const int mine = x[1];
        block_sums(x, total, warps);
        const int at = add_most(parts, x[1]);
        // Only where sequences claim the same rows (a cu_q that cannot be used) can there be more parts than room: those
        // behind are passed over.
        if (add_most(at, mine) > p.room) q_len = chunks = 0;
        if (b < B) {
            SharedSeq to = {};
            to.t0 = t0;
            to.q_len = q_len;
            to.kv_len = kv_len;
            to.row = b;
            to.page0 = group >= 0 ? start[group] >> p.page_log2 : 0;
            to.group = group;
            to.chunks = chunks;
            to.first_item = p.first[b] = add_most(items, x[0]);
            to.parts = at;
            p.own[b] = to;
        }
        items = add_most(items, total[0]);
        parts = add_most(parts, total[1]);
    }
    if (threadIdx.x == 0) {
        SharedHead head = {};
        head.items = p.first[B] = items;
        head.chunk = chunk;
        head.ctas = C;
        head.units = U;
        *p.head = head;
    }
    // ---- where the prompt kernel's CTAs begin
    __syncthreads();
#pragma unroll 1
    for (int c = threadIdx.x; c < p.ctas; c += T) {
        SharedWalk w = {};
        if (c < C) {
            const int u0 = whole ? c : shared_begin(c, U, C), g = last_at(length, G, u0);
            const int tiles = tiles_of(start[g]), split = active[g], per = whole ? split : tiles + kPOverShared;
            const int block = (u0 - length[g]) / per, at = u0 - length[g] - block * per;  // its place in the block
            const int blocks = blocks_of(tokens[g]) / p.heads;
            w.b = g;
            w.h = block / blocks;
            w.rb = block - w.h * blocks;
            w.t0 = row0[g];
            w.q_len = tokens[g];
            w.kv_len = start[g];
            w.tiles = tiles;
            w.tile = whole ? (int)((unsigned)at * tiles / split) : max(0, at - kPOverShared);
            w.left = whole ? kPOverShared + (int)((unsigned)(at + 1) * tiles / split) : shared_begin(c + 1, U, C) - u0 + at;
        }
        p.walks[c] = w;
    }
}
constexpr int kPlanBytes = (7 * kSharedMaxGroups + 1 + 4 * kPlanHeld) * 4;

// Joins the parts of eight (kJoinFew: four) rows of a sequence and kv head: a row a
// warp for the parts' factors and total, then the rows side by side, so that whole
// sectors are read from parts of either layout.  Latency bounds it: its parts (5 to
// 60 MB) come from L2, six (twelve) loads of a thread at a time; 5 to 7 us.
constexpr int kJoinThreads = 512, kJoinRows = 8, kJoinFew = 4;
constexpr int kJoinHeld = 192;  // parts of a row whose factors are kept: all of its group's, a CTA each
struct JoinRow {
    const float *own, *first, *rest;  // its sequence's chunks; its group's first part and those behind it
    int n_own, n_group;
    int values, quad;                 // of the group's parts: where values are, floats from four entries to the next four
    float inv, top;
};
template <int DP, int kRows>
__global__ void __launch_bounds__(kJoinThreads, kRows == kJoinFew ? 1 : 2) attn_shared_join_kernel(const SharedJoin p) {
    // A thread has four entries of a row; groups of threads take batches of parts in turn.
    constexpr int kGroup = kRows * DP / 4, kGroups = kJoinThreads / kGroup, kBatch = kRows == kJoinFew ? 12 : 6;
    __shared__ JoinRow row_of[kRows];
    __shared__ float factor[kRows][kJoinHeld];
    __shared__ float4 others[kGroups > 1 ? kGroup : 1];
    const int b = blockIdx.x / p.c.heads, h = blockIdx.x - b * p.c.heads, row0 = blockIdx.y * kRows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = p.c.d, width = d + 4;
    const long long rest_step = 2ll * p.slot_floats;  // of a block's CTAs but the first it is the first block
    griddep_wait();
    const SharedSeq s = p.own[b];
    const int C = p.head->ctas;
    const int U = p.head->units, rows = s.q_len * p.g;
    const long long own_step = (long long)rows * width;
    if (row0 >= rows) return;
    auto load = [](const float *x) { return __ldcg(reinterpret_cast<const float4 *>(x)); };
    if (warp < kRows && row0 + warp < rows) {
        const int r = row0 + warp;
        JoinRow x = {};
        nvfp4_in_bounds((long long)s.parts + (long long)s.chunks * rows * p.c.heads <= p.room, p.err);
        int stats = d;  // of the group's parts
        x.n_own = s.chunks;
        x.own = p.parts + (s.parts + (long long)h * s.chunks * rows + r) * width;
        x.quad = 4;
        if (s.group >= 0) {
            const SharedSeq pre = p.prefixes[s.group];
            const int i = r / p.g, rp = (s.t0 - pre.t0) * p.g + r;
            const int block = h * ((pre.q_len * p.g + kPRows - 1) / kPRows) + rp / kPRows, tiles = pre.kv_len / kPTile;
            const int ub = pre.units + block * (tiles + kPOverShared);  // its first unit
            const int ca = pre.split ? pre.units + block * pre.split : shared_owner(ub + kPOverShared, U, C);
            const int cb = pre.split ? ca + pre.split - 1 : shared_owner(ub + kPOverShared + tiles - 1, U, C);
            x.n_group = cb - ca + 1;
            if (!nvfp4_in_bounds(ca >= 0 && cb >= ca && cb < C && C <= p.ctas && rp >= 0 && rp < pre.q_len * p.g, p.err))
                x.n_group = 0;
            if (cb > ca) {
                const int rr = rp % kPRows;
                x.first = p.partials + ca * rest_step + (pre.split || shared_begin(ca, U, C) >= ub ? 0 : p.slot_floats);
                x.rest = p.partials + (ca + 1) * rest_step;
                stats = 4 * rr;
                x.values = 4 * kPRows + 4 * rr;
                x.quad = 4 * kPRows;
            } else {  // a block of one CTA has its part in a row's place
                x.first = p.rows + ((size_t)(s.t0 + i) * p.q.heads + h * p.g + r - i * p.g) * width;
            }
        }
        const int n = x.n_own + x.n_group;
        float top = -INFINITY, top_n = -INFINITY, sum = 0.f;
        for (int c = lane; c < n; c += 32) {  // its group's, then its sequence's
            const int k = c - x.n_group;
            const float4 y = load(k >= 0 ? x.own + k * own_step + d : (c == 0 ? x.first : x.rest + (c - 1) * rest_step) + stats);
            if (c < kJoinHeld) factor[warp][c] = y.x;
            top = fmaxf(top, y.x);
            const float m = fmaxf(top_n, y.y), at = m > -INFINITY ? m : 0.f;
            sum = fmaf(exp2_approx(top_n - at), sum, exp2_approx(y.y - at) * y.z);
            top_n = m;
        }
        float all_n = top_n;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            all_n = fmaxf(all_n, __shfl_xor_sync(0xffffffffu, all_n, o));
        }
        const bool any = all_n > -INFINITY;
        sum *= exp2_approx(top_n - (any ? all_n : 0.f));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        x.top = any ? top : 0.f;
        x.inv = attn_inverse(any ? top - all_n : 0.f, sum);
        for (int c = lane; c < min(n, kJoinHeld); c += 32) factor[warp][c] = exp2_approx(factor[warp][c] - x.top);
        if (lane == 0) row_of[warp] = x;
    }
    __syncthreads();
    const int local = threadIdx.x & (kRows - 1), r = row0 + local, group = threadIdx.x / kGroup;
    const int at4 = threadIdx.x / kRows & (DP / 4 - 1);  // these four entries of row r
    const bool here = r < rows && 4 * at4 < d;
    const JoinRow x = row_of[r < rows ? local : 0];
    // the gate, asked for before the sums
    const int i = r / p.g, hq = h * p.g + r - i * p.g;
    uint2 gate = make_uint2(0, 0);
    if (p.gate.p && group == 0 && here) {
        const uint16_t *const gp = p.gate.p + (s.t0 + i) * p.gate.ts + hq * p.gate.hs + 4 * at4;
        gate = p.gate.vec ? *reinterpret_cast<const uint2 *>(gp)
                          : make_uint2((uint32_t)gp[0] | (uint32_t)gp[1] << 16, (uint32_t)gp[2] | (uint32_t)gp[3] << 16);
    }
    const int n = here ? x.n_group + x.n_own : 0;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int c0 = group * kBatch; c0 < n; c0 += kGroups * kBatch) {
        float4 y[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int c = c0 + k;
            const bool own = c >= x.n_group;
            const float *const part = own ? x.own + (c - x.n_group) * own_step
                                          : (c == 0 ? x.first : x.rest + (c - 1) * rest_step) + x.values;
            y[k] = c < n ? load(part + at4 * (own ? 4 : x.quad)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int c = c0 + k;
            if (c >= n) break;
            const float w =
                c < kJoinHeld ? factor[local][c] : exp2_approx(__ldcg(x.own + (c - x.n_group) * own_step + d) - x.top);
            v.x = fmaf(w, y[k].x, v.x);
            v.y = fmaf(w, y[k].y, v.y);
            v.z = fmaf(w, y[k].z, v.z);
            v.w = fmaf(w, y[k].w, v.w);
        }
    }
    static_assert(kGroups <= 2, "one other group's sums are added");
    if constexpr (kGroups > 1) {
        if (group > 0) others[threadIdx.x % kGroup] = v;
        __syncthreads();
        if (group > 0) return;
        const float4 o = others[threadIdx.x];
        v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
    }
    if (!here) return;
    float y[4] = {v.x * x.inv, v.y * x.inv, v.z * x.inv, v.w * x.inv};
    if (p.gate.p && x.inv != 0.f) {  // (a row that saw no token is zero whatever its gate holds)
        y[0] *= sigmoid(__uint_as_float(gate.x << 16));
        y[1] *= sigmoid(__uint_as_float(gate.x & 0xFFFF0000u));
        y[2] *= sigmoid(__uint_as_float(gate.y << 16));
        y[3] *= sigmoid(__uint_as_float(gate.y & 0xFFFF0000u));
    }
    *reinterpret_cast<uint2 *>(p.y + ((size_t)(s.t0 + i) * p.q.heads + hq) * d + 4 * at4) =
        make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
}

}  // namespace

cudaError_t attn_shared_set_smem_limit() {
    return cudaFuncSetAttribute(attn_shared_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanBytes);
}

cudaError_t launch_attn_shared_plan(const SharedPlan &p, cudaStream_t stream) {
    const int most = p.groups + p.n.b < kPlanThreads ? (p.groups + p.n.b + 31) / 32 * 32 : kPlanThreads;
    return launch_behind(attn_shared_plan_kernel, dim3(1), most, kPlanBytes, stream, p);
}

cudaError_t launch_attn_shared_join(const SharedJoin &p, cudaStream_t stream) {
    const int rows = p.n.max_q * p.g, pairs = p.n.b * p.c.heads;
    auto grid = [&](int of_cta) { return dim3((unsigned)pairs, (unsigned)((rows + of_cta - 1) / of_cta)); };
    if (p.c.d <= 128) return launch_behind(attn_shared_join_kernel<128, kJoinRows>, grid(kJoinRows), kJoinThreads, 0, stream, p);
    // Heads of 256 entries: four rows a CTA, for a second group of threads and twice the loads in flight, where that makes
    // no more CTAs than SMs (16 sequences of 6 rows and 4 heads over 8192: 30.7 us; 34 with eight rows), else eight (64 such
    // over 2048: 33 us; 35 with four, as one wave of CTAs becomes two).
    return (long long)pairs * ((rows + kJoinFew - 1) / kJoinFew) <= p.ctas
               ? launch_behind(attn_shared_join_kernel<256, kJoinFew>, grid(kJoinFew), kJoinThreads, 0, stream, p)
               : launch_behind(attn_shared_join_kernel<256, kJoinRows>, grid(kJoinRows), kJoinThreads, 0, stream, p);
}

}  // namespace nvfp4
