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
// prefix as those of one sequence that sees all of it, and each sequence's with
// its own tokens, in whatever order and chunks; one kernel joins what they leave.
// The prefix is read once for 16 rows (attn_chunks.cu, few rows) or for 128
// (attn_prompt.cu, many) where each sequence for itself would read it again.
//
// What is shared of a prefix is what every token of the group sees, whole pages
// and whole tiles of 128 tokens of it: so it needs no masks, and what is left of
// it is read with each sequence's own tokens.
#include "attn.cuh"
#include "attn_units.h"

namespace nvfp4 {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kChunkUnit = 64;  // chunks are whole multiples of so many tokens

// Exclusive sum over the CTA's threads; *total is the sum of all.
__device__ __forceinline__ long long block_sum(long long x, long long *total, long long *warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warps[warp] = incl;
    __syncthreads();
    long long all = warps[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, all, o);
        if (lane >= o) all += v;
    }
    const long long before = __shfl_sync(0xffffffffu, all, (warp + 31) & 31);
    *total = __shfl_sync(0xffffffffu, all, 31);
    __syncthreads();
    return incl - x + (warp ? before : 0);
}

// One CTA: the records of groups and sequences.
__global__ void __launch_bounds__(kPlanThreads) attn_shared_plan_kernel(const SharedPlan p) {
    __shared__ int cu[kSharedMaxGroups + 1], start[kSharedMaxGroups], first[kSharedMaxGroups], active[kSharedMaxGroups];
    __shared__ long long warps[32];
    const int G = p.groups, B = p.n.b, unit = max(kPTile, 1 << p.page_log2);
    griddep_wait();
    griddep_launch_dependents();  // they wait for this kernel's end
    bool ok = true;
    for (int g = threadIdx.x; g <= G; g += kPlanThreads) {
        const int c = p.group_cu[g];
        cu[g] = c;
        if (g < G) {
            start[g] = first[g] = 0x7FFFFFFF;
            active[g] = 0;
            ok = ok && c >= 0 && p.group_cu[g + 1] >= c;
        } else {
            ok = ok && c <= B;
        }
    }
    ok = __syncthreads_and(ok);
    if (!ok && threadIdx.x == 0) atomicOr(p.err, kDevErrAttnInput);
    // The group of sequence b, -1 if it is in none.
    auto group_of = [&](int b) {
        if (!ok || b < cu[0] || b >= cu[G]) return -1;
        int lo = 0, hi = G;  // the last group that begins at b or before: empty ones come before it
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= b)
                lo = mid;
            else
                hi = mid;
        }
        return lo;
    };
    // ---- what all tokens of a group see
    bool neighbours = true;  // every row belongs to one sequence
    for (int b = threadIdx.x; b < B; b += kPlanThreads) {
        int t0, q_len, kv_len;
        const int g = group_of(b);
        if (!kv_sequence(p.n, b, &t0, &q_len, &kv_len)) atomicOr(p.err, kDevErrAttnInput);
        neighbours = neighbours && p.n.cu[b + 1] - p.n.cu[b] == q_len && (q_len == 0 || p.n.cu[b] == t0);
        if (g >= 0 && q_len > 0 && kv_len > 0) {  // others see nothing of the prefix
            atomicMin(&start[g], max(0, kv_len - q_len));
            atomicMin(&first[g], b);
            atomicAdd(&active[g], 1);
        }
    }
    neighbours = __syncthreads_and(neighbours);
    for (int g = threadIdx.x; g < G; g += kPlanThreads) {
        int shared = 0, t0 = 0, tokens = 0;
        if (ok && neighbours && active[g] > 1) {
            const int length = p.prefix_lens[g];
            shared = length > p.n.max_kv ? 0 : min(max(length, 0), start[g]) / unit * unit;
            if (shared > 0) {
                t0 = p.n.cu[cu[g]];
                tokens = p.n.cu[cu[g + 1]] - t0;
                if (tokens > p.max_group_tokens) shared = tokens = 0;
            }
        }
        if (ok && (p.prefix_lens[g] < 0 || p.prefix_lens[g] > p.n.max_kv)) atomicOr(p.err, kDevErrAttnInput);
        SharedSeq *const to = p.prefixes + g;
        to->t0 = t0;
        to->q_len = shared > 0 ? tokens : 0;
        to->kv_len = shared;
        to->row = shared > 0 ? first[g] : 0;
        to->page0 = 0;
        to->group = -1;
        start[g] = shared;
    }
    __syncthreads();
    // ---- all blocks of rows times their tokens, and all rows
    const int records = G + B;
    auto record = [&](int i, int *t0, int *q_len, int *kv_len, int *group) {  // of group i, or of sequence i - G
        if (i < G) {
            const SharedSeq *const s = p.prefixes + i;
            *t0 = s->t0;
            *q_len = s->q_len;
            *kv_len = s->kv_len;
            *group = -1;
        } else {
            kv_sequence(p.n, i - G, t0, q_len, kv_len);
            *group = *kv_len > 0 ? group_of(i - G) : -1;
            if (*group >= 0) {
                const int shared = start[*group];
                *kv_len -= shared;
                if (shared == 0) *group = -1;
            }
        }
    };
    auto blocks_of = [&](int q_len) { return (q_len * p.g + p.rows_chunk - 1) / p.rows_chunk; };
    long long work = 0, rows = 0;
    for (int i = threadIdx.x + (p.tensor ? G : 0); i < records; i += kPlanThreads) {
        int t0, q_len, kv_len, group;
        record(i, &t0, &q_len, &kv_len, &group);
        work += (long long)blocks_of(q_len) * p.heads * kv_len;
        rows += (long long)q_len * p.g * p.heads * kv_len;
    }
    long long all_work, all_rows;
    block_sum(work, &all_work, warps);
    block_sum(rows, &all_rows, warps);
    const long long by_items = (all_work + p.most_items - 1) / p.most_items;
    const long long by_floats = (all_rows * (p.d + 4) + p.most_floats - 1) / p.most_floats;
    const int chunk = (int)max(1ll, (max(by_items, by_floats) + kChunkUnit - 1) / kChunkUnit) * kChunkUnit;
    // ---- where each one's chunks, parts and units begin
    long long items = 0, floats = 0, units = 0;
    for (int i0 = 0; i0 < records; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        int t0 = 0, q_len = 0, kv_len = 0, group = -1, chunks = 0;
        long long mine = 0;
        if (i < records) {
            record(i, &t0, &q_len, &kv_len, &group);
            if (i >= G || !p.tensor)
                chunks = q_len > 0 ? (kv_len + chunk - 1) / chunk : 0;
            else if (q_len > 0)  // in the prompt kernel's units
                mine = (long long)((q_len * p.g + kPRows - 1) / kPRows) *
                       (prompt_block_tiles(p.g, q_len, kv_len, 0, false) + kPOver) * p.heads;
        }
        long long total;
        const long long part_floats = (long long)chunks * q_len * p.g * p.heads * (p.d + 4);
        const long long at = floats + block_sum(part_floats, &total, warps);
        floats += total;
        // Only where sequences claim the same rows (a cu_q that cannot be used) can there be more parts than room: those
        // behind are passed over.
        if (at + part_floats > p.room) q_len = chunks = 0;
        const long long item = items + block_sum((long long)chunks * blocks_of(q_len) * p.heads, &total, warps);
        items += total;
        const long long u = units + block_sum(mine, &total, warps);
        units += total;
        if (i < records) {
            SharedSeq *const to = i < G ? p.prefixes + i : p.own + (i - G);
            if (i >= G) {
                const int shared = group >= 0 ? start[group] : 0;
                to->t0 = t0;
                to->q_len = q_len;
                to->kv_len = kv_len;
                to->row = i - G;
                to->page0 = shared >> p.page_log2;
                to->group = group;
            }
            to->chunks = chunks;
            to->first_item = (int)item;
            to->floats = at;
            to->units = u;
            p.first[i] = (int)item;
        }
    }
    if (threadIdx.x == 0) {
        p.first[records] = (int)items;
        p.head->items = (int)items;
        p.head->chunk = chunk;
        p.head->units = units;
    }
}

// Joins the parts of eight rows of a sequence and kv head: a row a warp for the
// parts' factors and total, then the rows side by side, so that whole sectors
// are read from parts of either layout.
constexpr int kJoinThreads = 256, kJoinRows = 8;
template <int DP>
__global__ void __launch_bounds__(kJoinThreads) attn_shared_join_kernel(const SharedJoin p) {
    __shared__ float sh_m[kJoinRows], sh_inv[kJoinRows];
    griddep_wait();
    const int b = blockIdx.x / p.c.heads, h = blockIdx.x - b * p.c.heads, row0 = blockIdx.y * kJoinRows;
    const SharedSeq s = p.own[b];
    const int rows = s.q_len * p.g, d = p.c.d, width = d + 4;
    if (row0 >= rows) return;
    SharedSeq pre = {};
    if (s.group >= 0) pre = p.prefixes[s.group];
    const long long C = min((long long)p.ctas, p.head->units), U = p.head->units;
    // The parts of row r: its sequence's chunks, then its group's.
    struct Parts {
        const float *own, *pre;       // first chunk's
        long long own_step, pre_step; // floats from one to the next
        int n_own, n;
        int ca, rr;                   // the prompt kernel's: first CTA and row of its block; ca < 0: none
        long long ub;
    };
    auto parts_of = [&](int r) {
        Parts x = {};
        x.n = x.n_own = s.chunks;
        x.own = p.parts + s.floats + ((long long)h * s.chunks * rows + r) * width;
        x.own_step = (long long)rows * width;
        x.ca = -1;
        if (s.group < 0) return x;
        const int i = r / p.g, rp = (s.t0 - pre.t0) * p.g + r;
        if (p.tensor) {
            const int blocks = (pre.q_len * p.g + kPRows - 1) / kPRows;
            const int tiles = prompt_block_tiles(p.g, pre.q_len, pre.kv_len, 0, false);
            x.ub = pre.units + ((long long)h * blocks + rp / kPRows) * (tiles + kPOver);
            const int ca = (int)(((x.ub + kPOver + 1) * C - 1) / U), cb = (int)(((x.ub + kPOver + tiles) * C - 1) / U);
            if (cb > ca) {
                x.ca = ca;
                x.rr = rp % kPRows;
                x.n += cb - ca + 1;
            } else {
                x.pre = p.rows + ((size_t)(s.t0 + i) * p.q.heads + h * p.g + r - i * p.g) * width;
                x.n += 1;
            }
        } else {
            const int all = pre.q_len * p.g;
            x.pre = p.parts + pre.floats + ((long long)h * pre.chunks * all + rp) * width;
            x.pre_step = (long long)all * width;
            x.n += pre.chunks;
        }
        return x;
    };
    // Part c's stats, or (quad >= 0) four entries.
    auto at = [&](const Parts &x, int c, int quad) {
        if (c < x.n_own) return x.own + c * x.own_step + (quad < 0 ? d : 4 * quad);
        c -= x.n_own;
        if (x.ca < 0) return x.pre + c * x.pre_step + (quad < 0 ? d : 4 * quad);
        const float *const part = attn_part(p, x.ca + c, x.ub, U, C);
        return part + (quad < 0 ? 4 * x.rr : 4 * kPRows + (quad * kPRows + x.rr) * 4);
    };
    auto load = [](const float *x) { return __ldcg(reinterpret_cast<const float4 *>(x)); };
    {
        const int r = row0 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
        if (r < rows) {
            const Parts x = parts_of(r);
            float top = -INFINITY, top_n = -INFINITY;
            for (int c = lane; c < x.n; c += 32) {
                const float4 y = load(at(x, c, -1));
                top = fmaxf(top, y.x);
                top_n = fmaxf(top_n, y.y);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                top_n = fmaxf(top_n, __shfl_xor_sync(0xffffffffu, top_n, o));
            }
            const bool any = top_n > -INFINITY;
            float sum = 0.f;
            for (int c = lane; c < x.n; c += 32) {
                const float4 y = load(at(x, c, -1));
                sum = fmaf(exp2_approx(y.y - (any ? top_n : 0.f)), y.z, sum);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) {
                sh_m[r - row0] = any ? top : 0.f;
                sh_inv[r - row0] = attn_inverse(any ? top - top_n : 0.f, sum);
            }
        }
    }
    __syncthreads();
    const int r = row0 + (threadIdx.x & 7);
    if (r >= rows) return;
    const Parts x = parts_of(r);
    const float top = sh_m[r - row0], inv = sh_inv[r - row0];
    constexpr int kItems = DP / 128, kBatch = 8;
    const int quad = threadIdx.x >> 3;
    float4 v[kItems];
#pragma unroll
    for (int z = 0; z < kItems; ++z) v[z] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = 0; c0 < x.n; c0 += kBatch) {
        float4 y[kItems][kBatch];
        float f[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (c0 + k >= x.n) continue;
            f[k] = __ldcg(at(x, c0 + k, -1));
#pragma unroll
            for (int z = 0; z < kItems; ++z)
                if (4 * (quad + 32 * z) < d) y[z][k] = load(at(x, c0 + k, quad + 32 * z));
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (c0 + k >= x.n) continue;
            const float w = exp2_approx(f[k] - top);
#pragma unroll
            for (int z = 0; z < kItems; ++z) {
                v[z].x = fmaf(w, y[z][k].x, v[z].x);
                v[z].y = fmaf(w, y[z][k].y, v[z].y);
                v[z].z = fmaf(w, y[z][k].z, v[z].z);
                v[z].w = fmaf(w, y[z][k].w, v[z].w);
            }
        }
    }
#pragma unroll
    for (int z = 0; z < kItems; ++z) attn_store4(p, s.t0, h, r, rows, 4 * (quad + 32 * z), v[z], inv);
}

}  // namespace

cudaError_t launch_attn_shared_plan(const SharedPlan &p, cudaStream_t stream) {
    return launch_behind(attn_shared_plan_kernel, dim3(1), kPlanThreads, 0, stream, p);
}

cudaError_t launch_attn_shared_join(const SharedJoin &p, cudaStream_t stream) {
    const dim3 grid((unsigned)p.n.b * p.c.heads, (unsigned)((p.n.max_q * p.g + kJoinRows - 1) / kJoinRows));
    return p.c.d > 128 ? launch_behind(attn_shared_join_kernel<256>, grid, kJoinThreads, 0, stream, p)
                       : launch_behind(attn_shared_join_kernel<128>, grid, kJoinThreads, 0, stream, p);
}

}  // namespace nvfp4
