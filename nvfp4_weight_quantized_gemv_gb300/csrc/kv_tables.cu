// kv_tables.cu -- a step's block tables, slot map, positions and cumulative
// lengths from the requests' lengths and a ring of free pages.
//
// With want = kv + q and need = ceil(want / page) a sequence takes the pages
// [held, need) from the ring's head, or gives the pages [max(need, kept), held)
// back at its tail.  Where its pages and rows lie is a matter of exclusive sums
// over the batch: of the tokens and pages asked for (which decide who is
// served), of the pages given back, and of the tokens of those that are served.
//
// A few bytes a sequence and twelve a token: latency bounds it.  One launch of
// one cluster, whose CTAs all make the same sums for themselves (a scan over
// 1024 sequences is three times two barriers), share the pages and tokens, and
// meet once before anything that may be an input's own memory is written.
#include "batch_internal.h"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 1024;
constexpr int kCluster = 8;
constexpr int kAloneItems = 2048;

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
    long long all = warps[lane];  // every warp scans the warps' sums
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

// Last i of [0, n) with sums[i] <= x (sums[0] == 0, not decreasing).
__device__ __forceinline__ int owner(const int *sums, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// One CTA (kAlone) or a cluster of kCluster.
template <bool kAlone>
__global__ void __launch_bounds__(kThreads) kv_tables_kernel(const TablesParams p) {
    extern __shared__ int smem[];
    __shared__ long long warps[32];
    const int B = p.batch, log2 = p.page_log2;
    // by sequence: its first row, pages taken and given back by those before it, pages it holds from here on
    int *const cu = smem, *const take = cu + B + 1, *const back = take + B + 1, *const now = back + B + 1;
    const int rank = kAlone ? 0 : (int)cluster_ctarank();
    const int me = rank * kThreads + threadIdx.x, all = kAlone ? kThreads : kCluster * kThreads;
    griddep_wait();
    const long long head = p.span[0], tail = p.span[1];
    const bool span_ok = head >= 0 && tail >= head && tail - head <= p.ring;
    const long long free_pages = span_ok ? tail - head : 0;
    bool bad = !span_ok;

    // ---- who is served, and the sums
    long long asked = 0, grown = 0, given = 0;  // of the sequences so far
    int taken = 0, served = 0;                  // of those that are served
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        int kv = 0, q = 0, held = 0, kept = 0;
        if (b < B) {
            kv = p.kv[b];
            q = p.q[b];
            held = p.held[b];
            kept = p.kept ? p.kept[b] : 0;
        }
        const long long want = (long long)kv + q;
        bool ok = kv >= 0 && q >= 0 && kept >= 0 && kept <= held && held <= p.width && want <= ((long long)p.width << log2);
        bad |= !ok;
        long long total;
        const long long rows = asked + block_sum(ok ? q : 0, &total, warps) + q;
        asked += total;
        ok = ok && (q == 0 || rows <= p.tokens);
        const int need = ok ? (int)((want + (1 << log2) - 1) >> log2) : held;
        const int grow = max(0, need - held), less = ok ? max(0, held - max(need, kept)) : 0;
        const long long pages = grown + block_sum(grow, &total, warps);
        grown += total;
        ok = ok && (grow == 0 || pages + grow <= free_pages);
        const long long given_before = given + block_sum(less, &total, warps);
        given += total;
        const long long served_before = served + block_sum(ok ? q : 0, &total, warps);
        served += (int)total;
        block_sum(ok ? grow : 0, &total, warps);
        taken += (int)total;
        if (b < B) {
            cu[b] = (int)served_before;
            take[b] = (int)min(pages, free_pages);  // those who are served come before any who are not
            back[b] = (int)min(given_before, (long long)p.ring);
            now[b] = ok ? held + grow - less : held;
        }
    }
    const bool room = span_ok && free_pages + given <= p.ring;  // else some page is held twice: nothing is given back
    const int returned = room ? (int)given : 0;
    if (threadIdx.x == 0) {
        cu[B] = served;
        take[B] = taken;
        back[B] = returned;
    }
    if ((bad || !room) && rank == 0) atomicOr(p.err, kDevErrAttnInput);
    __syncthreads();
    const int at_head = span_ok ? (int)(head % p.ring) : 0, at_tail = span_ok ? (int)(tail % p.ring) : 0;
    auto from_ring = [&](int i) { return p.pages[at_head + i < p.ring ? at_head + i : at_head + i - p.ring]; };

    // ---- new pages, positions and slots
    for (int i = me; i < taken; i += all) {
        const int b = owner(take, B, i);
        p.table[b * p.table_stride + p.held[b] + i - take[b]] = from_ring(i);
    }
    for (int t = me; t < p.tokens; t += all) {
        int pos = 0;
        long long slot = -1;
        if (t < served) {
            const int b = owner(cu, B, t), held = p.held[b];
            pos = p.kv[b] + t - cu[b];
            const int pg = pos >> log2;
            const int page = pg < held ? p.table[b * p.table_stride + pg] : from_ring(take[b] + pg - held);
            slot = ((long long)page << log2) + (pos & ((1 << log2) - 1));
        }
        p.positions[t] = pos;
        p.slots[t] = slot;
    }
    // ---- what may lie in the inputs' own memory, after everybody has read them
    if (kAlone) {
        __syncthreads();
    } else {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    }
    for (int i = me; i < returned; i += all) {
        const int b = owner(back, B, i);
        const int page = p.table[b * p.table_stride + now[b] + i - back[b]];
        p.pages[at_tail + i < p.ring ? at_tail + i : at_tail + i - p.ring] = page;
    }
    for (int b = me; b < B; b += all) {
        const int kv = p.kv[b], held = p.held[b];
        p.cu[b] = cu[b];
        p.new_lens[b] = kv + cu[b + 1] - cu[b];
        p.held_out[b] = room ? now[b] : max(now[b], held);
    }
    if (me == 0) {
        p.cu[B] = served;
        p.span_out[0] = head + taken;
        p.span_out[1] = tail + returned;
    }
}

int tables_smem(int batch) { return (4 * batch + 3) * (int)sizeof(int); }

}  // namespace

cudaError_t tables_set_smem_limit() {
    cudaError_t e = cudaFuncSetAttribute(kv_tables_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         tables_smem(kTablesMaxBatch));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(kv_tables_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                tables_smem(kTablesMaxBatch));
}

cudaError_t launch_kv_tables(const TablesParams &p, cudaStream_t stream) {
    // Tokens and sequences that one CTA writes in a round or two need no cluster.
    if (p.tokens <= kAloneItems && p.batch <= kAloneItems)
        return launch_behind(kv_tables_kernel<true>, dim3(1), kThreads, tables_smem(p.batch), stream, p);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = tables_smem(p.batch);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kv_tables_kernel<false>, p);
}

}  // namespace nvfp4
