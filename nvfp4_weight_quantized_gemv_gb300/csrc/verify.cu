// verify.cu -- verification of drafted tokens against the target's
// probabilities, from given random numbers.
//
// Row i of a sequence is the target's distribution p_i of the token after the
// sequence's i-th.  The draft x_{i+1} is accepted while u_i q_i(x) < p_i(x); at
// the first row n that refuses its draft, or at the last row, the next token is
// drawn from r = max(p_n - q_n, 0), or from p_n: the smallest index at which the
// cumulative sum of r exceeds pick * sum(r).  So of all rows one is read whole,
// and HBM bounds it: two rows of `vocab` floats a sequence, or one.
//
// A cluster of eight CTAs a sequence (one for short vocabularies) shares the row
// in contiguous parts, a part a warp.  Sums are held in two fp32 numbers, their
// rounding errors and the differences' in the second one: to some 2^-46 of the sum
// (131072 entries of a softmax, or of the difference of two that are 0.5 to 1e-6 apart
// in their logits, at any scale: 2^-46 at most, mostly below 2^-52; Knuth's two-sum; fp64,
// two operations a clock on an SM here, took longer than the bytes).  CTAs push their warps' sums to all others and meet once; the
// part in which the sum passes the threshold is then read again by its CTA.  The
// sums and their order depend on the vocabulary and the rows' alignment alone.
//
// In a CUDA graph: one sequence of 32000 entries 6.8 us, all of it latency (the
// drafts' entries, the row, the cluster's barrier, the part); 64 of 131072 with 2 to 6
// rows each 19.6 us for 67 MB, 3.4 TB/s; 256 such 53 us, 5.1 TB/s.  (With lanes' sums that
// began at 1: 6.8, 19 and 52 us; then clusters of four, of 256 threads each, took 7.2 and
// 22 us, 256 sequences 49, those of 512 threads 8.1 and 20.)
#include "batch_internal.h"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCluster = 8;
// A CTA alone for short vocabularies, which a cluster's launch and barriers take longer than (us alone, in a cluster): 1 and 64
// sequences of 8192: 6.2 and 6.5, 6.7 and 10.5; of 16384: 7.8 and 6.8, 8.7 and 10.7; of 32000: 10.6 and 6.9, 13.6 and 11.1.
constexpr int kAloneVocab = 8192;
constexpr float kMostWeight = 1.8446744e19f;  // 2^64: sums of 2^31 entries are finite

// A number in two: h + l, |l| at most half a step of h.
struct Two {
    float h, l;
};
__device__ __forceinline__ Two two_of(float a, float b) {  // a + b, without error
    const float h = a + b, z = h - a;
    return Two{h, (a - (h - z)) + (b - z)};
}
__device__ __forceinline__ Two add(Two a, Two b) {
    const Two s = two_of(a.h, b.h), e = two_of(a.l, b.l);
    const Two x = two_of(s.h, s.l + e.h);
    return two_of(x.h, x.l + e.l);
}
__device__ __forceinline__ bool above(Two a, Two b) { return a.h > b.h || (a.h == b.h && a.l > b.l); }
__device__ __forceinline__ Two times(float x, Two a) {
    const float h = x * a.h;
    return two_of(h, fmaf(x, a.h, -h) + x * a.l);
}
__device__ __forceinline__ Two shuffle_xor(Two a, int o) {
    return Two{__shfl_xor_sync(0xffffffffu, a.h, o), __shfl_xor_sync(0xffffffffu, a.l, o)};
}
// Sum over a warp's lanes (or its first eight, ..) up to this one.
template <int kLanes>
__device__ __forceinline__ Two warp_scan(Two a) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int o = 1; o < kLanes; o <<= 1) {
        const Two v{__shfl_up_sync(0xffffffffu, a.h, o), __shfl_up_sync(0xffffffffu, a.l, o)};
        if (lane >= o) a = add(a, v);
    }
    return a;
}
__device__ __forceinline__ Two lane_before(Two a) {  // the lane before's, 0 for the first
    const Two v{__shfl_up_sync(0xffffffffu, a.h, 1), __shfl_up_sync(0xffffffffu, a.l, 1)};
    return threadIdx.x & 31 ? v : Two{0.f, 0.f};
}
__device__ __forceinline__ void st_cluster_two(uint32_t addr, Two x) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x.h), "f"(x.l) : "memory");
}

// The weight of an entry: p - q without error, 0 if that is no weight.
__device__ __forceinline__ Two weight(float p, float q) {
    const Two r = two_of(p, -q);
    return r.h > 0.f && r.h <= kMostWeight ? r : Two{0.f, 0.f};
}

// The sum of a lane's weights that are in flight together, none negative and `most`
// the largest: it begins at a power of two above that (and is exact when that is
// taken off again), so that a weight is never larger than what it is added to and
// its error takes two operations (Dekker's fast two-sum).  `error`: of the weights.
template <int N>
__device__ __forceinline__ Two batch_sum(const float (&x)[N], float most, float error) {
    const float begin = __uint_as_float((__float_as_uint(most) & 0x7F800000u) + 0x00800000u);
    float s = begin;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float t = s + x[i];
        error += x[i] - (t - s);
        s = t;
    }
    return two_of(s - begin, error);
}
// a + b for numbers that are not negative.
__device__ __forceinline__ Two add_positive(Two a, Two b) {
    const Two s = two_of(a.h, b.h);
    return two_of(s.h, s.l + (a.l + b.l));
}

// The rows whose entries are weighed: r = p - q, or p without q; entry `none` has no weight.
struct Row {
    const float *p, *q;
    int vocab, none;
    int lead;      // entries of group 0 before the row; groups of four are aligned in p's row
    int whole0, whole1;  // groups that the row fills
    bool wide;     // q's row is aligned likewise
};
// A lane's share of groups g0 .. g1 - 1.  Without kAny no r may be above the
// largest weight: `*most_of_all` tells whether one was.
template <bool kAny>
__device__ __forceinline__ Two sum_groups(const Row &row, int g0, int g1, float *most_of_all) {
    const int lane = threadIdx.x & 31;
    Two sum{0.f, 0.f};
    float over = 0.f;
    auto entry_off = [&](float4 &a, int g) {
        const int at = row.none - (4 * g - row.lead);
        if (row.none >= 0 && at >= 0 && at < 4) {
            if (at == 0) a.x = 0.f;
            if (at == 1) a.y = 0.f;
            if (at == 2) a.z = 0.f;
            if (at == 3) a.w = 0.f;
        }
    };
    constexpr int kPar = 8;  // groups of a lane in flight, half of them of q where there is one
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const int w1 = min(g1, row.whole1);
    int g = max(g0, row.whole0) + lane;
    const float4 *const p4 = reinterpret_cast<const float4 *>(row.p - row.lead);
    if (!row.q) {
#pragma unroll 1
        for (; g < w1; g += 32 * kPar) {
            float4 a[kPar];
            float x[4 * kPar], most = 0.f;
#pragma unroll
            for (int k = 0; k < kPar; ++k) a[k] = g + 32 * k < w1 ? p4[g + 32 * k] : zero;
#pragma unroll
            for (int k = 0; k < kPar; ++k) {
                entry_off(a[k], g + 32 * k);
                const float p[4] = {a[k].x, a[k].y, a[k].z, a[k].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[4 * k + i] = kAny ? weight(p[i], 0.f).h : fmaxf(p[i], 0.f);
                    most = fmaxf(most, x[4 * k + i]);
                }
            }
            over = fmaxf(over, most);
            sum = add_positive(sum, batch_sum(x, most, 0.f));
        }
    } else {
#pragma unroll 1
        for (; g < w1; g += 32 * (kPar / 2)) {
            float4 a[kPar / 2], b[kPar / 2];
            float x[2 * kPar], most = 0.f, error = 0.f;
#pragma unroll
            for (int k = 0; k < kPar / 2; ++k) {
                const int at = g + 32 * k;
                a[k] = b[k] = zero;
                if (at < w1) {
                    a[k] = p4[at];
                    const float *const b4 = row.q + 4 * at - row.lead;
                    b[k] = row.wide ? *reinterpret_cast<const float4 *>(b4) : make_float4(b4[0], b4[1], b4[2], b4[3]);
                }
            }
#pragma unroll
            for (int k = 0; k < kPar / 2; ++k) {
                entry_off(a[k], g + 32 * k);
                const float p[4] = {a[k].x, a[k].y, a[k].z, a[k].w}, q[4] = {b[k].x, b[k].y, b[k].z, b[k].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const Two r = kAny ? weight(p[i], q[i]) : two_of(p[i], -q[i]);
                    x[4 * k + i] = fmaxf(r.h, 0.f);
                    most = fmaxf(most, r.h);
                    if (r.h > 0.f) error += r.l;
                }
            }
            over = fmaxf(over, most);
            sum = add_positive(sum, batch_sum(x, most, error));
        }
    }
    // the row's ends: entries of groups that it does not fill
#pragma unroll 1
    for (int end = 0; end < 2; ++end) {
        const int at = end ? row.whole1 : 0;
        if (at < g0 || at >= g1 || (at >= row.whole0 && at < row.whole1) || (end && row.whole1 == 0)) continue;
        const int i = 4 * at - row.lead + lane;
        if (lane < 4 && i >= 0 && i < row.vocab)
            sum = add_positive(sum, weight(i == row.none ? 0.f : row.p[i], row.q ? row.q[i] : 0.f));
    }
    *most_of_all = over;
    return sum;
}

// (up to 64 registers: with no bound given the form of one CTA got 48, and spilled)
template <int kCtas>
__global__ void __launch_bounds__(kThreads, 4) verify_drafts_kernel(const VerifyParams p) {
    __shared__ __align__(8) Two sums[2][kCtas][kWarps];  // by pass: all CTAs' warps'
    __shared__ Two scan[kWarps];
    __shared__ int sh_n, sh_first, sh_last;
    const int rank = kCtas == 1 ? 0 : (int)cluster_ctarank(), b = blockIdx.x / kCtas;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_wait();
    const int t0 = p.cu[b], t1 = p.cu[b + 1];
    const int kv = p.kv ? p.kv[b] : 0;
    const bool usable = t0 >= 0 && t1 >= t0 && t1 <= p.rows;
    if (!usable || t1 == t0) {  // the whole cluster
        if (rank == 0 && threadIdx.x == 0) {
            if (!usable) atomicOr(p.err, kDevErrAttnInput);
            p.accepted[b] = 0;
            p.next[b] = -1;
            if (p.kv) p.new_lens[b] = kv;
        }
        return;
    }
    if (kCtas > 1) cluster_arrive();  // others' shared memory is written only once their CTAs run
    // ---- the accepted drafts
    const int drafts = t1 - t0 - 1;
    if (warp == 0) {
        int n = drafts;
        for (int i0 = 0; i0 < drafts; i0 += 32) {
            const int i = i0 + lane;
            bool yes = i >= drafts;
            if (!yes) {
                const int t = t0 + i, x = p.tokens[t + 1];
                const float u = p.u[t];
                if (x >= 0 && x < p.vocab) {
                    const float px = p.target[t * p.target_stride + x];
                    const float qx = p.draft ? p.draft[t * p.draft_stride + x] : 1.f;
                    yes = (double)u * (double)qx < (double)px;
                } else if (rank == 0) {
                    atomicOr(p.err, kDevErrAttnInput);
                }
            }
            const unsigned no = __ballot_sync(0xffffffffu, !yes);
            if (no) {
                n = i0 + __ffs(no) - 1;
                break;
            }
        }
        if (lane == 0) {
            sh_n = n;
            sh_first = 0x7FFFFFFF;
            sh_last = -1;
        }
    }
    __syncthreads();
    const int n = sh_n, row = t0 + n;
    const bool refused = n < drafts;
    const float *const pr = p.target + row * p.target_stride;
    const float *const qr = refused && p.draft ? p.draft + row * p.draft_stride : nullptr;
    const int hidden = refused && !p.draft ? p.tokens[row + 1] : -1;  // an entry that has no weight
    const float u = p.pick[b];
    const float pick = u >= 0.f ? u : 0.f;
    if (rank == 0)
        for (int i = threadIdx.x; i <= drafts; i += kThreads)
            if (i != n) p.out[t0 + i] = i < n ? p.tokens[t0 + i + 1] : -1;

    // ---- the weights' sums, in groups of four entries that are aligned in p's row, a contiguous run of groups a warp
    const int lead = (int)((reinterpret_cast<uintptr_t>(pr) >> 2) & 3);
    const int groups = (int)(((long long)p.vocab + lead + 3) >> 2);
    const int run = (groups + kCtas * kWarps - 1) / (kCtas * kWarps);
    Row rw{pr, qr, p.vocab, hidden, lead, lead ? 1 : 0, (p.vocab + lead) >> 2, false};
    rw.wide = qr && (int)((reinterpret_cast<uintptr_t>(qr) >> 2) & 3) == lead;
    for (int pass = 0; pass < 2; ++pass) {
        if (pass > 0) {  // p itself
            rw.q = nullptr;
            rw.none = -1;
        }
        auto entry = [&](int i) { return weight(i == rw.none ? 0.f : pr[i], rw.q ? rw.q[i] : 0.f); };
        const int g0 = min(groups, (rank * kWarps + warp) * run), g1 = min(groups, g0 + run);
        float most;
        Two part = sum_groups<false>(rw, g0, g1, &most);
        if (__any_sync(0xffffffffu, most > kMostWeight)) part = sum_groups<true>(rw, g0, g1, &most);
#pragma unroll 1
        for (int o = 16; o > 0; o >>= 1) part = add(part, shuffle_xor(part, o));
        if constexpr (kCtas == 1) {
            if (lane == 0) sums[pass][0][warp] = part;
            __syncthreads();
        } else {
            if (pass == 0) cluster_wait();
            if (lane < kCtas) st_cluster_two(cluster_map(smem_u32(&sums[pass][rank][warp]), (uint32_t)lane), part);
            __syncwarp();
            cluster_arrive();
            cluster_wait();
        }
        // ---- the CTA, then the warp, in whose part the sum passes the threshold
        static_assert(kWarps == 8 && (kCtas == 8 || kCtas == 1), "scans of eight lanes");
        auto find = [&](Two own, Two incl, Two before, Two limit, Two *begin) {  // eight lanes' sums, and up to each
            const Two x = add(before, incl), prev = lane_before(incl);
            const unsigned past = __ballot_sync(0xffffffffu, above(x, limit)) & 0xFF;
            // (not from differences of the sums up to each: those of lanes without weight differ in their rounding)
            const unsigned some = __ballot_sync(0xffffffffu, own.h > 0.f) & 0xFF;
            const int at = past & some ? __ffs(past & some) - 1 : 31 - __clz(some);
            const Two all = add(before, prev);
            *begin = Two{__shfl_sync(0xffffffffu, all.h, max(at, 0)), __shfl_sync(0xffffffffu, all.l, max(at, 0))};
            return at;  // -1: no part has any weight
        };
        auto limit_of = [&](Two all) { return pick < 1.f ? times(pick, all) : Two{INFINITY, 0.f}; };  // no sum is above that
        auto last_of = [&](Two a) { return Two{__shfl_sync(0xffffffffu, a.h, 7), __shfl_sync(0xffffffffu, a.l, 7)}; };
        int cta = 0;
        Two begin{0.f, 0.f}, total, limit;
        if constexpr (kCtas > 1) {
            // a CTA's eight sums by four lanes, its total to lane `CTA`
            const Two *const pair = &sums[pass][0][0] + 2 * lane;
            Two x = add(pair[0], pair[1]);
            x = add(x, shuffle_xor(x, 1));
            x = add(x, shuffle_xor(x, 2));
            x = Two{__shfl_sync(0xffffffffu, x.h, (lane & 7) * 4), __shfl_sync(0xffffffffu, x.l, (lane & 7) * 4)};
            if (lane >= 8) x = Two{0.f, 0.f};
            const Two incl = warp_scan<8>(x);
            total = last_of(incl);
            limit = limit_of(total);
            cta = max(0, find(x, incl, begin, limit, &begin));
        }
        const Two own_warp = lane < kWarps ? sums[pass][cta][lane & 7] : Two{0.f, 0.f}, incl_warps = warp_scan<8>(own_warp);
        if constexpr (kCtas == 1) {
            total = last_of(incl_warps);
            limit = limit_of(total);
        }
        if (!(total.h > 0.f)) {
            if (pass == 0 && refused) continue;  // p <= q everywhere: from p itself
            if (rank == 0 && threadIdx.x == 0) atomicOr(p.err, kDevErrAttnInput);
        }
        if (rank != cta) return;
        const int part_warp = max(0, find(own_warp, incl_warps, begin, limit, &begin));
        // ---- its entries, in order: a run of them a thread
        const int p0 = min(groups, (cta * kWarps + part_warp) * run), p1 = min(groups, p0 + run);
        const int e0 = max(0, 4 * p0 - lead), e1 = min(p.vocab, 4 * p1 - lead), per = (e1 - e0 + kThreads - 1) / kThreads;
        const int f0 = min(e1, e0 + (int)threadIdx.x * per), f1 = min(e1, f0 + per);
        Two here{0.f, 0.f};
        int last = -1;
        constexpr int kBatch = 8;
        auto each = [&](auto use) {  // use(entry, weight) is false: enough
#pragma unroll 1
            for (int i = f0; i < f1; i += kBatch) {
                Two w[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) w[k] = i + k < f1 ? entry(i + k) : Two{0.f, 0.f};
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    if (!use(i + k, w[k])) return;
            }
        };
        each([&](int i, Two w) {
            const Two t = two_of(here.h, w.h);
            here = Two{t.h, here.l + (t.l + w.l)};
            if (w.h > 0.f) last = i;
            return true;
        });
        here = two_of(here.h, here.l);
        // sum over the threads before
        const Two incl = warp_scan<32>(here);
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        Two at = begin;
        for (int w = 0; w < warp; ++w) at = add(at, scan[w]);
        at = add(at, lane_before(incl));
        if (last >= 0) {
            atomicMax(&sh_last, last);
            if (above(add(at, here), limit)) {
                int first = last;
                each([&](int i, Two w) {
                    at = add(at, w);
                    if (!(w.h > 0.f && above(at, limit))) return true;
                    first = i;
                    return false;
                });
                atomicMin(&sh_first, first);
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            const int token = max(0, sh_first < p.vocab ? sh_first : sh_last);
            p.accepted[b] = n;
            p.next[b] = token;
            p.out[row] = token;
            if (p.kv) p.new_lens[b] = kv - (drafts - n);
        }
        return;
    }
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyParams &p, cudaStream_t stream) {
    if (p.vocab <= kAloneVocab)
        return launch_behind(verify_drafts_kernel<1>, dim3((unsigned)p.batch), kThreads, 0, stream, p);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.batch * kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_drafts_kernel<kCluster>, p);
}

}  // namespace nvfp4
