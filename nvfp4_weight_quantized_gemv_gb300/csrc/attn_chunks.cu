// attn_chunks.cu -- attention over the paged 8-bit cache, a chunk of tokens and
// up to 16 query rows a warp, for batches that share prefixes.
//
// A warp takes its chunk's tokens 16 at a time, from memory straight into the
// registers that mma.sync reads them from:
//
//     S^T = K Q^T (tokens x rows),   O^T += V^T P^T (entries x rows),
//
// with the codes made f16 (exactly) on the way, and the softmax kept per row as
// in the kernel for few rows: w = s + log2 vscale(page), m the running maximum
// of w and n that of s, the product's weights 2^(w - m + 8) and the total's
// 2^(s - n), both references left as they are until a weight would pass 2^15.
// The chunk's result, (O, m, n, total) of each row, is a part that another
// kernel joins with the others of its rows.
//
// Why a warp, and no shared memory.  What a sequence holds behind its prefix is
// short: a CTA of eight warps in rings and teams spends as long on a block's
// queries, the merge of its warps and the wait for its first tile as on its tokens
// (64 sequences of 510 to 1021 tokens, 32 + 8 heads of 128: 32 us for 100 MB).
// Warps of their own have nothing to wait for but their loads, and 8 to 16 of
// them an SM keep 32 to 64 KB of those in flight.  A step's K is asked for as soon
// as the last one's has been multiplied, its V likewise, so that one set of
// registers each suffices.  Rows of a prefix in blocks of 16 are neighbouring
// warps, which find the chunk in L1.
#include "attn.cuh"

namespace nvfp4 {

namespace {

constexpr int kStep = 16;                   // tokens of a step: of one page
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr float kWeightSlack = 7.f;         // weights are 2^kWeightLift at the maximum and at most 2^7 above
constexpr float kSumSlack = 60.f;

__device__ __forceinline__ uint32_t nan_bytes(uint32_t v) { return ((v & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

template <int DP, int NT>
struct Chunk {
    static constexpr bool kQShared = NT > 1;  // query fragments in shared memory
    static constexpr int kQ = kQShared ? DP / 16 * NT * 32 * 8 : 0;
    static constexpr int kWarpBytes = kQ + DP * 4;  // and first tokens whose values are NaN, by entry
    static constexpr int kBytes = kWarps * kWarpBytes;
    // warps that the registers leave room for
    static constexpr int kCtas = DP == 128 && NT == 1 ? 2 : 1;
};

// The rows [row0, row0 + 8 NT) of record s and kv head h over tokens [from, to).
template <int DP, int NT>
__device__ __forceinline__ void run_chunk(const ChunkParams &p, const SharedSeq &s, bool causal, int h, int row0, int from,
                                          int to, float *part, uint2 *sq, int *nan_from) {
    constexpr int kHalves = DP / 128, kSteps = DP / 16;
    constexpr bool kQShared = NT > 1;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rows = s.q_len * p.g, d = p.c.d;
    const int start = causal ? s.kv_len - s.q_len : s.kv_len;
    const int *const pages = p.n.table + (size_t)s.row * p.n.table_stride + s.page0;

    // ---- pages of the next 32 steps, a lane each: where the step's codes begin (-1: reads as zeros) and its scales
    long long offset = -1;
    float kscale = 1.f, vlog = 0.f;
    auto look_up = [&](int tok) {
        tok += lane * kStep;
        offset = -1;
        kscale = 1.f;
        vlog = 0.f;
        if (tok < to) {
            const int page = pages[tok >> p.c.page_log2];
            if (page < 0 || page >= p.c.pages) {
                atomicOr(p.err, kDevErrAttnInput);
            } else {
                offset = page * p.c.ps + h * p.c.hs + (tok & (p.c.page - 1)) * p.c.ts;
                kscale = p.c.ks[(size_t)page * p.c.heads + h];
                vlog = log2f(p.c.vs[(size_t)page * p.c.heads + h]);
            }
        }
    };
    look_up(from);
    uint4 kf[2 * kHalves][2], vf[kHalves][4];
    auto load_k = [&](long long at) {
        const uint8_t *const a = p.c.k + at + g * p.c.ts + 16 * t;
#pragma unroll
        for (int i = 0; i < 2 * kHalves; ++i) {
            const bool on = at >= 0 && i * 64 + 16 * t < d;
            kf[i][0] = on ? *reinterpret_cast<const uint4 *>(a + i * 64) : make_uint4(0, 0, 0, 0);
            kf[i][1] = on ? *reinterpret_cast<const uint4 *>(a + i * 64 + 8 * p.c.ts) : make_uint4(0, 0, 0, 0);
        }
    };
    auto load_v = [&](long long at) {
        const uint8_t *const a = p.c.v + at + 2 * t * p.c.ts + 16 * g;
#pragma unroll
        for (int i = 0; i < kHalves; ++i) {
            const bool on = at >= 0 && i * 128 + 16 * g < d;
#pragma unroll
            for (int z = 0; z < 4; ++z)
                vf[i][z] = on ? *reinterpret_cast<const uint4 *>(a + i * 128 + ((z & 1) + (z >> 1) * 8) * p.c.ts)
                              : make_uint4(0, 0, 0, 0);
        }
    };
    {
        const long long at = __shfl_sync(0xffffffffu, offset, 0);
        load_k(at);
        load_v(at);
    }

    // ---- the query rows as B fragments, each scaled by a power of two to a maximum in [2^7, 2^8)
    uint2 qf[kQShared ? 1 : kSteps];
    float qs[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        uint32_t u[kSteps][2];  // bf16 pairs, then f16 pairs
        const int r = row0 + 8 * n + g;
        const bool on = r < rows;
        const int i = on ? p.g_div(r) : 0, hq = h * p.g + (on ? r - i * p.g : 0);
        const uint16_t *const src = p.q.p + (s.t0 + i) * p.q.ts + hq * p.q.hs;
        uint32_t two = 0;
#pragma unroll
        for (int k = 0; k < kSteps; k += 4) {  // 16 entries of this lane
            const int e = k * 16 + 16 * t;
            uint4 a = make_uint4(0, 0, 0, 0), b = a;
            if (on && e < d) {
                a = load_rows8(src + e, p.q.vec);
                b = load_rows8(src + e + 8, p.q.vec);
            }
            u[k][0] = a.x, u[k][1] = a.y, u[k + 1][0] = a.z, u[k + 1][1] = a.w;
            u[k + 2][0] = b.x, u[k + 2][1] = b.y, u[k + 3][0] = b.z, u[k + 3][1] = b.w;
#pragma unroll
            for (int w = 0; w < 4; ++w) two = __vmaxu2(two, __vmaxu2(u[k + w][0] & 0x7FFF7FFFu, u[k + w][1] & 0x7FFF7FFFu));
        }
        int most = (int)max(two & 0xFFFFu, two >> 16);  // the largest magnitude's bits
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
        const int ex = most > 0 ? min(max((most >> 7) - 127 - 7, -119), 119) : 0;
        const float down = pow2i(-ex);
        // a row that is not finite has no scores
        const float scale = most < 0x7F80 ? pow2i(ex) * p.scale_log2 : __int_as_float(0x7FC00000);
#pragma unroll
        for (int c = 0; c < 2; ++c) qs[n][c] = __shfl_sync(0xffffffffu, scale, (2 * t + c) * 4);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const __half2 x = __floats2half2_rn(__uint_as_float(u[k][w] << 16) * down,
                                                    __uint_as_float(u[k][w] & 0xFFFF0000u) * down);
                u[k][w] = *reinterpret_cast<const uint32_t *>(&x);
            }
            if constexpr (kQShared)
                sq[(k * NT + n) * 32 + lane] = make_uint2(u[k][0], u[k][1]);
            else
                qf[k] = make_uint2(u[k][0], u[k][1]);
        }
    }
    if constexpr (kQShared) __syncwarp();

    float o[kHalves * 8][NT][4], m[NT][2], ns[NT][2], l[NT][2];
    int lim[NT][2];  // last token that the row sees
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int r = row0 + 8 * n + 2 * t + c;
            lim[n][c] = r < rows ? start + p.g_div(r) : -1;
            m[n][c] = ns[n][c] = -INFINITY;
            l[n][c] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < kHalves * 8; ++k)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[k][n][c] = 0.f;
    }
    // tokens that every row, that any row sees
    const int all_see = max(0, start + p.g_div(row0) + 1), some_see = s.kv_len;
    bool some_nan = false;

    int left = 32;  // steps that the lanes have looked up
    for (int tok = from; tok < to; tok += kStep) {
        const int now = (32 - left) & 31;
        const float ks = __shfl_sync(0xffffffffu, kscale, now), lvs = __shfl_sync(0xffffffffu, vlog, now);
        if (--left == 0) {
            left = 32;
            look_up(tok + kStep);
        }
        const long long next = __shfl_sync(0xffffffffu, offset, (32 - left) & 31);
        const bool more = tok + kStep < to;
        // ---- scores
        float s0[NT][4], s1[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) s0[n][c] = s1[n][c] = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * kHalves; ++i) {
            const uint32_t w0[4] = {kf[i][0].x, kf[i][0].y, kf[i][0].z, kf[i][0].w};
            const uint32_t w1[4] = {kf[i][1].x, kf[i][1].y, kf[i][1].z, kf[i][1].w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t a0, a1, a2, a3;
                e4m3x4_f16(w0[w], a0, a2);
                e4m3x4_f16(w1[w], a1, a3);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint2 q = kQShared ? sq[((i * 4 + w) * NT + n) * 32 + lane] : qf[kQShared ? 0 : i * 4 + w];
                    mma_f16(w & 1 ? s1[n] : s0[n], a0, a1, a2, a3, q.x, q.y);
                }
            }
        }
        if (more) load_k(next);
        // ---- softmax
        const bool edge = tok + kStep > all_see;  // some row does not see some token
        bool grow = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float f = qs[n][c] * ks;
                s0[n][c] = (s0[n][c] + s1[n][c]) * f;
                s0[n][2 + c] = (s0[n][2 + c] + s1[n][2 + c]) * f;
                if (edge) {
                    if (tok + g > lim[n][c]) s0[n][c] = -INFINITY;
                    if (tok + g + 8 > lim[n][c]) s0[n][2 + c] = -INFINITY;
                }
                const float x = fmaxf(s0[n][c], s0[n][2 + c]);
                grow |= x + lvs > m[n][c] + kWeightSlack || x > ns[n][c] + kSumSlack;
            }
        }
        if (__any_sync(0xffffffffu, grow)) {  // the rows' maxima over all lanes, only where they matter
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float f[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float y = fmaxf(s0[n][c], s0[n][2 + c]);
#pragma unroll
                    for (int o2 = 4; o2 < 32; o2 *= 2) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o2));
                    f[c] = 1.f;
                    // (a row's references depend on its own scores alone)
                    if (y + lvs > m[n][c] + kWeightSlack || y > ns[n][c] + kSumSlack) {
                        const float x = fmaxf(m[n][c], y + lvs);
                        y = fmaxf(ns[n][c], y);
                        f[c] = exp2_approx(m[n][c] - x);
                        l[n][c] *= exp2_approx(ns[n][c] - y);
                        m[n][c] = x;
                        ns[n][c] = y;
                    }
                }
#pragma unroll
                for (int k = 0; k < kHalves * 8; ++k) {
                    o[k][n][0] *= f[0];
                    o[k][n][1] *= f[1];
                    o[k][n][2] *= f[0];
                    o[k][n][3] *= f[1];
                }
            }
        }
        uint32_t pf[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float e[4];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const bool any = ns[n][c] > -INFINITY;  // else every weight is 0, or NaN
                const float ref = any ? m[n][c] - lvs - kWeightLift : 0.f, ref_l = any ? ns[n][c] : 0.f;
                e[c] = exp2_approx(s0[n][c] - ref);
                e[2 + c] = exp2_approx(s0[n][2 + c] - ref);
                l[n][c] += exp2_approx(s0[n][c] - ref_l) + exp2_approx(s0[n][2 + c] - ref_l);
            }
            const __half2 x = __floats2half2_rn(e[0], e[1]), y = __floats2half2_rn(e[2], e[3]);
            pf[n][0] = transpose8x8(*reinterpret_cast<const uint32_t *>(&x));
            pf[n][1] = transpose8x8(*reinterpret_cast<const uint32_t *>(&y));
        }
        // ---- values
        if (edge) {
            // A zero weight does not hide a NaN: codes that nobody sees become zeros, a NaN that only some rows
            // see is noted by entry and token (rows see all tokens from one on).
#pragma unroll
            for (int i = 0; i < kHalves; ++i)
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int at = tok + 2 * t + (z & 1) + (z >> 1) * 8;
                    uint32_t *const w = reinterpret_cast<uint32_t *>(&vf[i][z]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (at >= some_see) w[j] = 0;
                        const uint32_t bad = nan_bytes(w[j]);
                        if (bad && at >= all_see) {
                            some_nan = true;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (bad >> (8 * e) & 0x80u) {
                                    atomicMin(&nan_from[i * 128 + 16 * g + 4 * j + e], at);
                                    w[j] &= ~(0xFFu << (8 * e));
                                }
                        }
                    }
                }
        }
#pragma unroll
        for (int i = 0; i < kHalves; ++i) {
            const uint32_t va[4] = {vf[i][0].x, vf[i][0].y, vf[i][0].z, vf[i][0].w};
            const uint32_t vb[4] = {vf[i][1].x, vf[i][1].y, vf[i][1].z, vf[i][1].w};
            const uint32_t vc[4] = {vf[i][2].x, vf[i][2].y, vf[i][2].z, vf[i][2].w};
            const uint32_t vd[4] = {vf[i][3].x, vf[i][3].y, vf[i][3].z, vf[i][3].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint32_t sel = y ? 0x7362u : 0x5140u;
                    uint32_t a0, a1, a2, a3;
                    e4m3x4_f16(__byte_perm(va[j], vb[j], sel), a0, a1);
                    e4m3x4_f16(__byte_perm(vc[j], vd[j], sel), a2, a3);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_f16(o[i * 8 + 2 * j + y][n], a0, a1, a2, a3, pf[n][0], pf[n][1]);
                }
            }
        }
        if (more) load_v(next);
    }

    // ---- the part
    some_nan = __any_sync(0xffffffffu, some_nan);
    __syncwarp();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float x = l[n][c];
            x += __shfl_xor_sync(0xffffffffu, x, 4);
            x += __shfl_xor_sync(0xffffffffu, x, 8);
            x += __shfl_xor_sync(0xffffffffu, x, 16);
            const int r = row0 + 8 * n + 2 * t + c;
            if (r >= rows) continue;
            float *const to_row = part + (size_t)r * (d + 4);
            if (g == 0) *reinterpret_cast<float4 *>(to_row + d) = make_float4(m[n][c], ns[n][c], x, 0.f);
#pragma unroll
            for (int i = 0; i < kHalves; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int e = i * 128 + 16 * g + 4 * j, k = i * 8 + 2 * j;
                    if (e >= d) continue;
                    float4 y = make_float4(o[k][n][c], o[k][n][2 + c], o[k + 1][n][c], o[k + 1][n][2 + c]);
                    if (some_nan) {  // entries that are NaN from some token on
                        if (lim[n][c] >= nan_from[e]) y.x = __int_as_float(0x7FC00000);
                        if (lim[n][c] >= nan_from[e + 1]) y.y = __int_as_float(0x7FC00000);
                        if (lim[n][c] >= nan_from[e + 2]) y.z = __int_as_float(0x7FC00000);
                        if (lim[n][c] >= nan_from[e + 3]) y.w = __int_as_float(0x7FC00000);
                    }
                    *reinterpret_cast<float4 *>(to_row + e) = y;
                }
        }
    if (some_nan) {  // for the next chunk
        __syncwarp();
        for (int e = lane; e < DP; e += 32) nan_from[e] = 0x7FFFFFFF;
        __syncwarp();
    }
}

// Last i of [0, n) with sums[i] <= x, by a warp (sums[0] == 0, not decreasing).
__device__ __forceinline__ int owner_of(const int *sums, int n, int x) {
    const int lane = threadIdx.x & 31;
    int lo = 0;
    while (n > 1) {  // [lo, lo + n)
        const int step = (n + 31) / 32, at = min(lane * step, n);
        const bool below = at < n && __ldcg(sums + lo + at) <= x;
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, below));
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo;
}

template <int DP, int NT>
__global__ void __launch_bounds__(kThreads, Chunk<DP, NT>::kCtas) attn_chunks_kernel(const ChunkParams p) {
    extern __shared__ uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *const mine = smem + warp * Chunk<DP, NT>::kWarpBytes;
    uint2 *const sq = reinterpret_cast<uint2 *>(mine);
    int *const nan_from = reinterpret_cast<int *>(mine + Chunk<DP, NT>::kQ);
    for (int e = lane; e < DP; e += 32) nan_from[e] = 0x7FFFFFFF;
    __syncwarp();
    griddep_wait();
    const int items = p.head->items, size = p.head->chunk;
    for (int item = blockIdx.x * kWarps + warp; item < items; item += gridDim.x * kWarps) {
        const int record = owner_of(p.first, p.records, item);
        const SharedSeq s = p.seqs[record];
        // numbered by kv head, chunk and block of rows
        const int blocks = (s.q_len * p.g + 8 * NT - 1) / (8 * NT), i = item - s.first_item;
        const int c = i / blocks, row0 = (i - c * blocks) * 8 * NT, h = c / s.chunks, chunk = c - h * s.chunks;
        const int from = chunk * size, to = min(s.kv_len, from + size);
        float *const part = p.parts + s.floats + (long long)c * (s.q_len * p.g) * (p.c.d + 4);
        const bool causal = record >= p.prefixes;
        if (NT > 1 && s.q_len * p.g - row0 <= 8)
            run_chunk<DP, 1>(p, s, causal, h, row0, from, to, part, sq, nan_from);
        else
            run_chunk<DP, NT>(p, s, causal, h, row0, from, to, part, sq, nan_from);
    }
}

template <int DP, int NT>
cudaError_t chunks_launch(const ChunkParams &p, cudaStream_t stream) {
    const int bytes = Chunk<DP, NT>::kBytes;
    static_assert(Chunk<DP, NT>::kBytes * Chunk<DP, NT>::kCtas <= 200 * 1024, "shared memory");
    if (bytes > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(attn_chunks_kernel<DP, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
    }
    return launch_behind(attn_chunks_kernel<DP, NT>, dim3((unsigned)(p.ctas * Chunk<DP, NT>::kCtas)), kThreads, (size_t)bytes,
                         stream, p);
}

}  // namespace

int attn_chunk_rows(int, int rows) { return rows <= 8 ? 8 : 16; }

cudaError_t launch_attn_chunks(const ChunkParams &p, int rows, cudaStream_t stream) {
    if (p.c.d > 128) return rows <= 8 ? chunks_launch<256, 1>(p, stream) : chunks_launch<256, 2>(p, stream);
    return rows <= 8 ? chunks_launch<128, 1>(p, stream) : chunks_launch<128, 2>(p, stream);
}

}  // namespace nvfp4
