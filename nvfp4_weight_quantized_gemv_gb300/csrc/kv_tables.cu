// kv_tables.cu -- a step's block tables, slot map, positions and cumulative
// lengths from the requests' lengths and a ring of free pages.
//
// With want = kv + q and need = ceil(want / page) a sequence takes the pages
// [held, need) from the ring's head, or gives the pages [max(need, kept), held)
// back at its tail.  Where its pages and rows lie is a matter of exclusive sums
// over the batch: of the tokens and pages asked for (which decide who is
// served), of the pages given back, and of the tokens of those that are served.
//
// A few bytes a sequence and twelve a token: latency bounds it (in a CUDA graph 4.3
// us for 16 sequences, 10 for 1024 with 28000 tokens).  One launch of
// one CTA, or for more of a cluster, whose CTAs all make the same sums for
// themselves, share the pages and tokens, and meet once before anything that may
// be an input's own memory is written.
#include "batch_internal.h"
#include "ptx.cuh"
#include "scan.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 1024;
constexpr int kCluster = 8;
// One CTA for so many tokens and sequences together: either way a CTA makes all sums, and what a cluster's others take over
// is the writing of both (us alone, in a cluster): one token of 512 sequences 5.3 and 6.6, of 1024 7.4 and 7.9, of 1280 10.7
// and 10.6, of 2048 11.3 and 10.8, of 4096 18.6 and 16.6; 5 tokens of 400 7.0 and 7.4, of 500 7.4 and 7.4, of 800 8.3 and
// 7.8; 20 of 125 6.7 and 6.9, of 150 7.3 and 7.2; 8 tokens of 2048 sequences in all 9.1 and 9.3, of 4096 15.4 and 15.0.
constexpr int kAloneItems = 2560;

// One CTA (kAlone) or a cluster of kCluster.
template <bool kAlone>
__global__ void __launch_bounds__(kThreads) kv_tables_kernel(const TablesParams p) {
    extern __shared__ int smem[];
    __shared__ int warps[2][32];
    __shared__ int sh_at[2];  // where in the ring the free pages begin and end
    const int B = p.batch, log2 = p.page_log2;
    // by sequence: its first row, pages taken and given back by those before it, pages it holds from here on and until
    // here, position of row 0 if that were its own
    int *const cu = smem, *const take = cu + B + 1, *const back = take + B + 1, *const now = back + B + 1,
        *const until = now + B, *const origin = until + B;
    const int rank = kAlone ? 0 : (int)cluster_ctarank();
    const int T = blockDim.x, me = rank * T + threadIdx.x, all = kAlone ? T : kCluster * T;
    griddep_wait();
    const long long head = p.span[0], tail = p.span[1];
    const bool span_ok = head >= 0 && tail >= head && tail - head <= p.ring;
    const int free_pages = span_ok ? (int)(tail - head) : 0;
    if (threadIdx.x < 2) sh_at[threadIdx.x] = span_ok ? (int)((threadIdx.x ? tail : head) % p.ring) : 0;
    bool bad = !span_ok;

    // ---- who is served, and the sums
    int asked = 0, grown = 0, given = 0, taken = 0, served = 0;  // of the sequences so far; the last two of those served
#pragma unroll 1
    for (int b0 = 0; b0 < B; b0 += T) {
        const int b = b0 + threadIdx.x;
        int kv = 0, q = 0, held = 0, kept = 0;
        if (b < B) {
            kv = p.kv[b];
            q = p.q[b];
            held = p.held[b];
            kept = p.kept ? p.kept[b] : 0;
        }
        const long long want = (long long)kv + q;
        bool ok = kv >= 0 && q >= 0 && kept >= 0 && kept <= held && held <= p.width && want <= ((long long)p.width << log2) &&
                  want <= kMost;  // (lengths and positions have 32 bits; a row may have pages for more)
        bad |= !ok;
        int x[1] = {ok ? q : 0}, all_x[1];
        block_sums(x, all_x, warps);
        ok = ok && (q == 0 || add_most(add_most(asked, x[0]), q) <= p.tokens);
        asked = add_most(asked, all_x[0]);
        const int need = ok ? (int)((want + (1 << log2) - 1) >> log2) : held;
        const int grow = max(0, need - held), less = ok ? max(0, held - max(need, kept)) : 0;
        int y[2] = {grow, less}, all_y[2];
        block_sums(y, all_y, warps);
        const int pages = add_most(grown, y[0]), given_before = add_most(given, y[1]);
        ok = ok && (grow == 0 || add_most(pages, grow) <= free_pages);
        grown = add_most(grown, all_y[0]);
        given = add_most(given, all_y[1]);
        int z[2] = {ok ? q : 0, ok ? grow : 0}, all_z[2];
        block_sums(z, all_z, warps);
        if (b < B) {
            cu[b] = served + z[0];
            take[b] = min(pages, free_pages);  // those who are served come before any who are not
            back[b] = min(given_before, p.ring);
            now[b] = ok ? held + grow - less : held;
            until[b] = held;
            origin[b] = (int)((unsigned)kv - (unsigned)cu[b]);
        }
        served += all_z[0];
        taken += all_z[1];
    }
    const bool room = span_ok && free_pages <= p.ring - min(given, p.ring);  // else some page is held twice: none is given back
    const int returned = room ? given : 0;
    if (threadIdx.x == 0) {
        cu[B] = served;
        take[B] = taken;
        back[B] = returned;
    }
    if ((bad || !room) && rank == 0) atomicOr(p.err, kDevErrAttnInput);
    __syncthreads();
    const int at_head = sh_at[0], at_tail = sh_at[1];
    auto from_ring = [&](int i) { return p.pages[at_head + i < p.ring ? at_head + i : at_head + i - p.ring]; };

    // ---- new pages, positions and slots
    for (int i = me; i < taken; i += all) {
        const int b = last_at(take, B, i);
        p.table[b * p.table_stride + until[b] + i - take[b]] = from_ring(i);
    }
    constexpr int kPar = 4;  // tokens of a thread that are looked up together
#pragma unroll 1
    for (int t0 = me; t0 < p.tokens; t0 += kPar * all) {
        int seq[kPar], page[kPar];
#pragma unroll
        for (int k = 0; k < kPar; ++k) seq[k] = 0;
#pragma unroll 1
        for (int n = B; n > 1;) {  // the last sequence that begins at or before the token
            const int half = n >> 1;
#pragma unroll
            for (int k = 0; k < kPar; ++k)
                if (cu[min(seq[k] + half, B)] <= t0 + k * all) seq[k] += half;
            n -= half;
        }
#pragma unroll
        for (int k = 0; k < kPar; ++k) {
            const int t = t0 + k * all, b = seq[k];
            page[k] = 0;
            if (t < served) {
                const int pg = (origin[b] + t) >> log2;
                page[k] = pg < until[b] ? p.table[b * p.table_stride + pg] : from_ring(take[b] + pg - until[b]);
            }
        }
#pragma unroll
        for (int k = 0; k < kPar; ++k) {
            const int t = t0 + k * all, pos = t < served ? origin[seq[k]] + t : 0;
            if (t >= p.tokens) break;
            p.positions[t] = pos;
            p.slots[t] = t < served ? ((long long)page[k] << log2) + (pos & ((1 << log2) - 1)) : -1;
        }
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
        const int b = last_at(back, B, i);
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

int tables_smem(int batch) { return (6 * batch + 3) * (int)sizeof(int); }

}  // namespace

cudaError_t tables_set_smem_limit() {
    cudaError_t e = cudaFuncSetAttribute(kv_tables_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         tables_smem(kTablesMaxBatch));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(kv_tables_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                tables_smem(kTablesMaxBatch));
}

cudaError_t launch_kv_tables(const TablesParams &p, cudaStream_t stream) {
    // Few tokens and sequences need no cluster, and a barrier of few warps is quick.
    if (p.tokens + p.batch <= kAloneItems) {
        const int most = p.tokens > p.batch ? p.tokens : p.batch, threads = most < kThreads ? (most + 31) / 32 * 32 : kThreads;
        return launch_behind(kv_tables_kernel<true>, dim3(1), threads > 0 ? threads : 32, tables_smem(p.batch), stream, p);
    }
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
