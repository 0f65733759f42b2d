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
// What is shared of a prefix is what every token of the group sees, whole pages
// and whole tiles of 128 tokens of it: so it needs no masks, and what is left of
// it is read with each sequence's own tokens.
#include "attn.cuh"
#include "attn_units.h"

namespace nvfp4 {

namespace {

constexpr int kPlanThreads = 1024;  // at most
constexpr int kChunkUnit = 64;      // chunks are whole multiples of so many tokens
constexpr int kPlanHeld = 1024;     // sequences whose lengths the plan keeps in shared memory

// Exclusive sums of N numbers over the CTA's threads, in place; total[i] is all threads'.
template <int N>
__device__ __forceinline__ void block_sums(long long (&x)[N], long long (&total)[N], long long (*warps)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, all = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        long long incl = x[i];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) warps[i][warp] = incl;
        x[i] = incl - x[i];
        total[i] = 0;
    }
    __syncthreads();
    for (int w = 0; w < all; ++w)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (w < warp) x[i] += warps[i][w];
            total[i] += warps[i][w];
        }
    __syncthreads();
}

// Last i of [0, n) with at[i] <= x.
template <class T, class U>
__device__ __forceinline__ int last_at(const T *at, int n, U x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// One CTA: the records of groups and sequences.  What it reads is asked for at
// once; the rest is arithmetic and a few barriers, 3 us of a call's chain.
__global__ void __launch_bounds__(kPlanThreads) attn_shared_plan_kernel(const SharedPlan p) {
    constexpr int kG = kSharedMaxGroups;
    extern __shared__ long long plan_smem[];
    __shared__ long long warps[3][32];
    // by group: first sequence; tokens that all see, then those that are shared; first sequence that holds some; such
    // sequences; first row and rows; first unit of the prompt kernel's
    long long *const units = plan_smem;
    int *const cu = reinterpret_cast<int *>(units + kG + 1), *const start = cu + kG + 1, *const first = start + kG,
        *const active = first + kG, *const row0 = active + kG, *const tokens = row0 + kG, *const length = tokens + kG;
    // by sequence, for the first kPlanHeld: first row, rows, tokens
    int *const s_t0 = length + kG, *const s_q = s_t0 + kPlanHeld, *const s_kv = s_q + kPlanHeld;
    const int G = p.groups, B = p.n.b, unit = max(kPTile, 1 << p.page_log2), T = blockDim.x;
    griddep_wait();
    bool ok = true, neighbours = true;  // neighbours: every row belongs to one sequence
    for (int b = threadIdx.x; b < B; b += T) {
        int t0, q_len, kv_len;
        if (!kv_sequence(p.n, b, &t0, &q_len, &kv_len)) atomicOr(p.err, kDevErrAttnInput);
        neighbours = neighbours && p.n.cu[b + 1] - p.n.cu[b] == q_len && (q_len == 0 || p.n.cu[b] == t0);
        if (b < kPlanHeld) {
            s_t0[b] = t0;
            s_q[b] = q_len;
            s_kv[b] = kv_len;
        }
    }
    for (int g = threadIdx.x; g <= G; g += T) {
        const int c = p.group_cu[g];
        cu[g] = c;
        if (g < G) {
            length[g] = p.prefix_lens[g];
            start[g] = first[g] = 0x7FFFFFFF;
            active[g] = 0;
            ok = ok && c >= 0 && p.group_cu[g + 1] >= c;
            if (length[g] < 0 || length[g] > p.n.max_kv) {
                atomicOr(p.err, kDevErrAttnInput);
                length[g] = 0;
            }
        } else {
            ok = ok && c <= B;
        }
    }
    ok = __syncthreads_and(ok);
    neighbours = __syncthreads_and(neighbours);
    if (!ok && threadIdx.x == 0) atomicOr(p.err, kDevErrAttnInput);
    // (what is nobody's group is behind no prefix; of groups that begin at one sequence all but the last are empty)
    auto group_of = [&](int b) { return !ok || b < cu[0] || b >= cu[G] ? -1 : last_at(cu, G, b); };
    auto sequence = [&](int b, int *t0, int *q_len, int *kv_len) {
        if (b < kPlanHeld) {
            *t0 = s_t0[b];
            *q_len = s_q[b];
            *kv_len = s_kv[b];
        } else {
            kv_sequence(p.n, b, t0, q_len, kv_len);
        }
    };
    // ---- what all tokens of a group see
    for (int b = threadIdx.x; b < B; b += T) {
        int t0, q_len, kv_len;
        const int g = group_of(b);
        sequence(b, &t0, &q_len, &kv_len);
        if (g >= 0 && q_len > 0 && kv_len > 0) {  // others see nothing of the prefix
            atomicMin(&start[g], max(0, kv_len - q_len));
            atomicMin(&first[g], b);
            atomicAdd(&active[g], 1);
        }
    }
    __syncthreads();
    for (int g = threadIdx.x; g < G; g += T) {
        int shared = 0, from = 0, rows = 0;
        if (ok && neighbours && active[g] > 1) {
            int t0, q_len, kv_len;
            sequence(cu[g + 1] - 1, &t0, &q_len, &kv_len);
            shared = min(length[g], start[g]) / unit * unit;
            from = p.n.cu[cu[g]];
            rows = p.n.cu[cu[g + 1]] - from;
            if (rows > p.max_group_tokens) shared = 0;
        }
        start[g] = shared;
        row0[g] = shared > 0 ? from : 0;
        tokens[g] = shared > 0 ? rows : 0;
    }
    __syncthreads();
    const int records = G + B;
    auto record = [&](int i, int *t0, int *q_len, int *kv_len, int *group) {  // of group i, or of sequence i - G
        *group = -1;
        if (i < G) {
            *t0 = row0[i];
            *q_len = tokens[i];
            *kv_len = start[i];
        } else {
            sequence(i - G, t0, q_len, kv_len);
            const int g = *kv_len > 0 ? group_of(i - G) : -1;
            if (g >= 0 && start[g] > 0) {
                *kv_len -= start[g];
                *group = g;
            }
        }
    };
    auto blocks_of = [&](int q_len) { return (q_len * p.g + p.rows_chunk - 1) / p.rows_chunk; };
    auto units_of = [&](int q_len, int kv_len) {  // of a group, in the prompt kernel's count
        return q_len == 0 ? 0ll : (long long)((q_len * p.g + kPRows - 1) / kPRows) *
                                      (prompt_block_tiles(p.g, q_len, kv_len, 0, false) + kPOver) * p.heads;
    };
    // ---- all blocks of rows times their own tokens, and all rows: how long a chunk is
    long long sum[3] = {0, 0, 0}, all[3];
    for (int i = threadIdx.x; i < records; i += T) {
        int t0, q_len, kv_len, group;
        record(i, &t0, &q_len, &kv_len, &group);
        if (i < G) {
            sum[2] += units_of(q_len, kv_len);
        } else {
            sum[0] += (long long)blocks_of(q_len) * p.heads * kv_len;
            sum[1] += (long long)q_len * p.g * p.heads * kv_len;
        }
    }
    block_sums(sum, all, warps);
    const long long by_items = div_small(all[0] + p.most_items - 1, p.most_items);
    const long long by_floats = div_small(all[1] * (p.d + 4) + p.most_floats - 1, p.most_floats);
    const int chunk = (int)max(1ll, (max(by_items, by_floats) + kChunkUnit - 1) / kChunkUnit) * kChunkUnit;
    // The prompt kernel's CTAs.  A unit of it costs as much as 12 steps of 16 tokens (heads of at most 128 entries: 1.1 us
    // of an SM, and 4 KB at its share of the memory's rate), or 8 (1.45 us and 8 KB).
    const float steps = (float)all[0] / 16.f, cost = (float)all[2] * (p.d <= 128 ? 12.f : 8.f);
    const long long U = all[2];
    const int share = (int)(p.ctas * (cost / fmaxf(cost + steps, 1.f)) + 0.5f);
    const int C = (int)min(U, (long long)max(1, steps > 0.f ? min(share, p.ctas - 1) : p.ctas));
    // ---- where each one's chunks, parts and units begin
    long long done[3] = {0, 0, 0};  // items, floats, units
    for (int i0 = 0; i0 < records; i0 += T) {
        const int i = i0 + threadIdx.x;
        int t0 = 0, q_len = 0, kv_len = 0, group = -1, chunks = 0;
        long long x[3] = {0, 0, 0}, total[3], room = 0;
        if (i < records) {
            record(i, &t0, &q_len, &kv_len, &group);
            if (i >= G) {
                chunks = q_len > 0 ? (kv_len + chunk - 1) / chunk : 0;
                x[0] = (long long)chunks * blocks_of(q_len) * p.heads;
                x[1] = room = (long long)chunks * q_len * p.g * p.heads * (p.d + 4);
            } else {
                x[2] = units_of(q_len, kv_len);
            }
        }
        block_sums(x, total, warps);
        if (i < records) {
            // Only where sequences claim the same rows (a cu_q that cannot be used) can there be more parts than room:
            // those behind are passed over.
            if (done[1] + x[1] + room > p.room) q_len = chunks = 0;
            SharedSeq to;
            to.t0 = t0;
            to.q_len = q_len;
            to.kv_len = kv_len;
            to.row = i < G ? (q_len > 0 ? first[i] : 0) : i - G;
            to.page0 = group >= 0 ? start[group] >> p.page_log2 : 0;
            to.group = group;
            to.chunks = chunks;
            to.first_item = (int)(done[0] + x[0]);
            to.floats = done[1] + x[1];
            to.units = done[2] + x[2];
            to.pad[0] = to.pad[1] = to.pad[2] = to.pad[3] = 0;
            if (i < G) {
                p.prefixes[i] = to;
                units[i] = to.units;
            } else {
                p.own[i - G] = to;
                p.first[i - G] = to.first_item;
            }
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) done[k] += total[k];
    }
    if (threadIdx.x == 0) {
        SharedHead head;
        head.items = (int)done[0];
        head.chunk = chunk;
        head.next = 0;
        head.ctas = C;
        head.units = U;
        head.pad[0] = head.pad[1] = 0;
        *p.head = head;
        p.first[B] = (int)done[0];
    }
    // ---- where the prompt kernel's CTAs begin
    __syncthreads();
    for (int c = threadIdx.x; c < p.ctas; c += T) {
        SharedWalk w = {};
        if (c < C) {
            const long long u0 = div_small(c * U, C), u1 = div_small((c + 1) * U, C);
            const int g = last_at(units, G, u0);
            const int blocks = (tokens[g] * p.g + kPRows - 1) / kPRows;
            const int tiles = prompt_block_tiles(p.g, tokens[g], start[g], 0, false), per = tiles + kPOver;
            const long long block = div_small(u0 - units[g], per), at = units[g] + block * per;
            w.b = g;
            w.h = (int)div_small(block, blocks);
            w.rb = (int)(block - (long long)w.h * blocks);
            w.tile = (int)max(0ll, u0 - at - kPOver);
            w.t0 = row0[g];
            w.q_len = tokens[g];
            w.kv_len = start[g];
            w.tiles = tiles;
            w.left = u1 - at;
        }
        p.walks[c] = w;
    }
}
constexpr int kPlanBytes = (kSharedMaxGroups + 1) * 8 + (7 * kSharedMaxGroups + 1 + 3 * kPlanHeld) * 4;

// Joins the parts of eight rows of a sequence and kv head: a row a warp for the
// parts' factors and total, then the rows side by side, so that whole sectors
// are read from parts of either layout.
constexpr int kJoinThreads = 256, kJoinRows = 8;
constexpr int kJoinHeld = 192;  // parts of a row whose factors are kept: all of its group's, a CTA each
struct JoinRow {
    const float *own, *first, *rest;  // its sequence's chunks; its group's first part and those behind it
    int n_own, n_group;
    int values, quad;                 // of the group's parts: where values are, floats from four entries to the next four
    float inv, top;
};
template <int DP>
__global__ void __launch_bounds__(kJoinThreads) attn_shared_join_kernel(const SharedJoin p) {
    __shared__ JoinRow row_of[kJoinRows];
    __shared__ float factor[kJoinRows][kJoinHeld];
    const int b = blockIdx.x / p.c.heads, h = blockIdx.x - b * p.c.heads, row0 = blockIdx.y * kJoinRows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = p.c.d, width = d + 4;
    const long long rest_step = 2ll * p.slot_floats;  // of a block's CTAs but the first it is the first block
    griddep_wait();
    const SharedSeq s = p.own[b];
    const int C = p.head->ctas;
    const long long U = p.head->units;
    const int rows = s.q_len * p.g;
    const long long own_step = (long long)rows * width;
    if (row0 >= rows) return;
    auto load = [](const float *x) { return __ldcg(reinterpret_cast<const float4 *>(x)); };
    if (row0 + warp < rows) {
        const int r = row0 + warp;
        JoinRow x = {};
        int stats = d;  // of the group's parts
        x.n_own = s.chunks;
        x.own = p.parts + s.floats + ((long long)h * s.chunks * rows + r) * width;
        x.quad = 4;
        if (s.group >= 0) {
            const SharedSeq pre = p.prefixes[s.group];
            const int i = r / p.g, rp = (s.t0 - pre.t0) * p.g + r;
            const int blocks = (pre.q_len * p.g + kPRows - 1) / kPRows, tiles = prompt_block_tiles(p.g, pre.q_len, pre.kv_len, 0, false);
            const long long ub = pre.units + ((long long)h * blocks + rp / kPRows) * (tiles + kPOver);
            const int ca = (int)div_small((ub + kPOver + 1) * C - 1, U), cb = (int)div_small((ub + kPOver + tiles) * C - 1, U);
            x.n_group = cb - ca + 1;
            if (cb > ca) {
                const int rr = rp % kPRows;
                x.first = p.partials + ca * rest_step + (div_small(ca * U, C) >= ub ? 0 : p.slot_floats);
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
    const int local = threadIdx.x & 7, r = row0 + local, quad = threadIdx.x >> 3;
    if (r >= rows) return;
    const JoinRow x = row_of[local];
    constexpr int kItems = DP / 128, kBatch = DP == 128 ? 8 : 6;
    float4 v[kItems];
#pragma unroll
    for (int z = 0; z < kItems; ++z) v[z] = make_float4(0.f, 0.f, 0.f, 0.f);
    // n parts, part c at at(c) and weighed with factor(c): four entries out of every 32 times `quads` floats.
    auto sum_parts = [&](int n, int quads, auto at, auto weight) {
        for (int c0 = 0; c0 < n; c0 += kBatch) {
            float4 y[kItems][kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
#pragma unroll
                for (int z = 0; z < kItems; ++z)
                    y[z][k] = c0 + k < n && 4 * (quad + 32 * z) < d ? load(at(c0 + k) + (quad + 32 * z) * quads)
                                                                    : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (c0 + k >= n) break;
                const float w = weight(c0 + k);
#pragma unroll
                for (int z = 0; z < kItems; ++z) {
                    v[z].x = fmaf(w, y[z][k].x, v[z].x);
                    v[z].y = fmaf(w, y[z][k].y, v[z].y);
                    v[z].z = fmaf(w, y[z][k].z, v[z].z);
                    v[z].w = fmaf(w, y[z][k].w, v[z].w);
                }
            }
        }
    };
    const float *const f = factor[local];
    sum_parts(
        x.n_group, x.quad, [&](int c) { return (c == 0 ? x.first : x.rest + (c - 1) * rest_step) + x.values; },
        [&](int c) { return f[c]; });
    const int held = min(x.n_own, kJoinHeld - x.n_group);
    sum_parts(
        held, 4, [&](int c) { return x.own + c * own_step; }, [&](int c) { return f[x.n_group + c]; });
    if (held < x.n_own)
        sum_parts(
            x.n_own - held, 4, [&](int c) { return x.own + (held + c) * own_step; },
            [&](int c) { return exp2_approx(__ldcg(x.own + (held + c) * own_step + d) - x.top); });
#pragma unroll
    for (int z = 0; z < kItems; ++z) attn_store4(p, s.t0, h, r, rows, 4 * (quad + 32 * z), v[z], x.inv);
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
    const dim3 grid((unsigned)p.n.b * p.c.heads, (unsigned)((p.n.max_q * p.g + kJoinRows - 1) / kJoinRows));
    return p.c.d > 128 ? launch_behind(attn_shared_join_kernel<256>, grid, kJoinThreads, 0, stream, p)
                       : launch_behind(attn_shared_join_kernel<128>, grid, kJoinThreads, 0, stream, p);
}

}  // namespace nvfp4
