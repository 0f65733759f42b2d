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
// in contiguous parts, a part a warp.  Sums are exact to about 2^-48: a lane adds
// in two fp32 numbers (the sum and its rounding errors, by Knuth's two-sum, the
// differences' errors too), warps and CTAs in fp64; fp64 alone, at this chip's
// rate, would cost more than the bytes.  CTAs push their sums to all others and
// meet once; the part in which the sum passes the threshold is then read again
// by its CTA, 256 threads with a scan in fp64.  The sums and their order depend on
// the vocabulary alone, and so does the token.
#include "batch_internal.h"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kAloneVocab = 4096;          // a CTA's 16 entries a thread
constexpr float kMostWeight = 1.8446744e19f;  // 2^64: sums of 2^31 entries are finite

__device__ __forceinline__ void st_cluster_f64(uint32_t addr, double x) {
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(x) : "memory");
}

// A sum in two fp32 numbers.
struct Sum2 {
    float s = 0.f, e = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float t = s + x, z = t - s;
        e += (s - (t - z)) + (x - z);
        s = t;
    }
};

// The weight of an entry, without its rounding error and that error.
__device__ __forceinline__ float weight(float p, float q, float *error) {
    const float r = p - q;
    if (!(r > 0.f && r <= kMostWeight)) {
        *error = 0.f;
        return 0.f;
    }
    const float z = r - p;
    *error = (p - (r - z)) - (q + z);
    return r;
}
__device__ __forceinline__ double weight64(float p, float q) {
    const float r = p - q;
    return r > 0.f && r <= kMostWeight ? (double)p - (double)q : 0.0;
}

// Exclusive sum over the CTA's threads, in their order.
__device__ __forceinline__ double block_sum(double x, double *warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    double incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warps[warp] = incl;
    __syncthreads();
    double before = 0.0;
    for (int w = 0; w < warp; ++w) before += warps[w];
    const double prev = __shfl_up_sync(0xffffffffu, incl, 1);
    return before + (lane ? prev : 0.0);
}

template <int kCtas>
__global__ void __launch_bounds__(kThreads) verify_drafts_kernel(const VerifyParams p) {
    __shared__ double sums[2][kCtas][kWarps];  // by pass: all CTAs' warps'
    __shared__ double scan[kWarps];
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
    const double pick = u >= 0.f ? (double)u : 0.0;
    if (rank == 0)
        for (int i = threadIdx.x; i <= drafts; i += kThreads)
            if (i != n) p.out[t0 + i] = i < n ? p.tokens[t0 + i + 1] : -1;

    // ---- the weights' sums.  Entries are taken in aligned groups of four, a contiguous run of groups a warp.
    const int lead = (int)((reinterpret_cast<uintptr_t>(pr) >> 2) & 3);  // entries of group 0 before the row
    const bool wide = !qr || (int)((reinterpret_cast<uintptr_t>(qr) >> 2) & 3) == lead;
    const int groups = (int)(((long long)p.vocab + lead + 3) >> 2);
    const int run = (groups + kCtas * kWarps - 1) / (kCtas * kWarps);
    // Group g of a row whose group 0 is aligned (or of one that is not: `aligned` false); zeros outside the row.
    auto load4 = [&](const float *r, int g, bool aligned) {
        const int i = 4 * g - lead;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i >= 0 && i <= p.vocab - 4) {
            if (aligned) return *reinterpret_cast<const float4 *>(r + i);
            return make_float4(r[i], r[i + 1], r[i + 2], r[i + 3]);
        }
        if (i >= 0 && i < p.vocab) v.x = r[i];
        if (i + 1 >= 0 && i + 1 < p.vocab) v.y = r[i + 1];
        if (i + 2 >= 0 && i + 2 < p.vocab) v.z = r[i + 2];
        if (i + 3 < p.vocab) v.w = r[i + 3];
        return v;
    };
    for (int pass = 0; pass < 2; ++pass) {
        const bool less = pass == 0 && qr;  // q is taken off
        const int none = pass == 0 ? hidden : -1;
        auto load_p = [&](int g) {
            float4 v = load4(pr, g, true);
            const int i = none - (4 * g - lead);
            if (none >= 0 && i >= 0 && i < 4) reinterpret_cast<float *>(&v)[i] = 0.f;
            return v;
        };
        auto load_q = [&](int g) { return less ? load4(qr, g, wide) : make_float4(0.f, 0.f, 0.f, 0.f); };
        const int g0 = min(groups, (rank * kWarps + warp) * run), g1 = min(groups, g0 + run);
        Sum2 sum;
        constexpr int kPar = 4;  // groups of a lane in flight
        for (int g = g0 + lane; g < g1; g += 32 * kPar) {
            float4 x[kPar], y[kPar];
#pragma unroll
            for (int k = 0; k < kPar; ++k) {
                x[k] = y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (g + 32 * k < g1) {
                    x[k] = load_p(g + 32 * k);
                    y[k] = load_q(g + 32 * k);
                }
            }
#pragma unroll
            for (int k = 0; k < kPar; ++k) {
                const float a[4] = {x[k].x, x[k].y, x[k].z, x[k].w}, c[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float error;
                    sum.add(weight(a[j], c[j], &error));
                    sum.e += error;
                }
            }
        }
        double part = (double)sum.s + (double)sum.e;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
        if constexpr (kCtas == 1) {
            if (lane == 0) sums[pass][0][warp] = part;
            __syncthreads();
        } else {
            if (pass == 0) cluster_wait();
            if (lane < kCtas) st_cluster_f64(cluster_map(smem_u32(&sums[pass][rank][warp]), (uint32_t)lane), part);
            __syncwarp();
            cluster_arrive();
            cluster_wait();
        }
        // ---- the CTA, then the warp, in whose part the sum passes the threshold
        auto find = [&](double x, double before, double limit, double *begin) {  // lanes' parts in order
            double incl = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            const unsigned past = __ballot_sync(0xffffffffu, before + incl > limit), some = __ballot_sync(0xffffffffu, x > 0.0);
            const int at = past & some ? __ffs(past & some) - 1 : 31 - __clz(some);
            const double to = __shfl_sync(0xffffffffu, incl, (at + 31) & 31);
            *begin = before + (at > 0 ? to : 0.0);
            return at;  // -1: no part has any weight
        };
        double mine = 0.0;
        if (lane < kCtas)
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mine += sums[pass][lane][w];
        double total = mine;
#pragma unroll
        for (int o = kCtas / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        total = __shfl_sync(0xffffffffu, total, 0);
        if (!(total > 0.0)) {
            if (pass == 0 && refused) continue;  // p <= q everywhere: from p itself
            if (rank == 0 && threadIdx.x == 0) atomicOr(p.err, kDevErrAttnInput);
        }
        const double limit = pick * total;
        double begin;
        const int cta = max(0, find(mine, 0.0, limit, &begin));
        if (rank != cta) return;
        const int part_warp = max(0, find(lane < kWarps ? sums[pass][cta][lane < kWarps ? lane : 0] : 0.0, begin, limit, &begin));
        // ---- its entries, in order: a run of groups a thread
        const int p0 = min(groups, (cta * kWarps + part_warp) * run), p1 = min(groups, p0 + run);
        const int per = (run + kThreads - 1) / kThreads;
        const int f0 = min(p1, p0 + (int)threadIdx.x * per), f1 = min(p1, f0 + per);
        auto each = [&](auto take) {  // take(entry, weight) is false: enough
            for (int g = f0; g < f1; ++g) {
                const float4 x = load_p(g), y = load_q(g);
                const float a[4] = {x.x, x.y, x.z, x.w}, c[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (!take(4 * g - lead + j, weight64(a[j], c[j]))) return;
            }
        };
        double here = 0.0;
        int last = -1;
        each([&](int i, double w) {
            here += w;
            if (w > 0.0) last = i;
            return true;
        });
        double at = begin + block_sum(here, scan);
        if (last >= 0) {
            atomicMax(&sh_last, last);
            if (at + here > limit) {
                int first = last;
                each([&](int i, double w) {
                    at += w;
                    if (!(w > 0.0 && at > limit)) return true;
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
