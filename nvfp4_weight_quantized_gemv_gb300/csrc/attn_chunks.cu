// attn_chunks.cu -- attention over the paged 8-bit cache, a chunk of tokens and
// up to 16 query rows a warp, for batches that share prefixes.
//
// A warp takes its chunk's tokens 16 at a time, in the layout that mma.sync reads
// registers in:
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
// What bounds it: memory, and before that latencies.  What a sequence holds
// behind its prefix is short: a CTA of eight warps that work on one block in rings
// and teams spends as long on the block's queries, the merge of its warps and the
// wait for its first tile as on the tokens (64 sequences of 510 to 1021 tokens, 32 +
// 8 heads of 128: 32 us for 100 MB).  A warp of its own waits for its own loads
// alone: its lanes copy the 16-byte pieces that they will read themselves (cp.async)
// into a ring of the warp's, two or three steps deep, 4 or 8 KB each.  Eight to
// sixteen warps an SM so keep 64 to 128 KB in flight, and no barrier is needed.  In
// that case 72 SMs take 40 us for them beside the prompt kernel, their schedulers busy
// for two thirds of it: 70 % of a warp's time are its steps, of 370 instructions a 16
// tokens with all that is around them.
//
// Chunks are of one length for the whole call, and warps take them in order from
// one counter: the next one's number is asked for while one is worked on.  A chunk
// costs 4 to 5 us besides its steps (its record, pages, scales and queries, one after
// the other), and a CTA's first ones another 3 (heads of 128) to 7 us (256), as an SM
// fetches the instructions.  So the best is one chunk for each warp, all taken at once,
// if their lengths allow for it; else several in turns.
#include "attn.cuh"

namespace nvfp4 {

namespace {

constexpr int kStep = 16;                   // tokens of a step: of one page
constexpr float kWeightSlack = 7.f;         // weights are 2^kWeightLift at the maximum and at most 2^7 above
constexpr float kSumSlack = 60.f;

__device__ __forceinline__ uint32_t nan_bytes(uint32_t v) { return ((v & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// 16 bytes into shared memory, zeros if `size` is 0 and not 16.
__device__ __forceinline__ void copy16(uint32_t to, const uint8_t *from, int size) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(size) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // until at most N groups are in flight
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int DP, int NT>
struct Chunk {
    static constexpr int kStages = DP == 128 ? 3 : 2;
    static constexpr int kStage = kStep * DP * 2;            // K and V of a step
    static constexpr bool kQShared = NT > 1;                 // query fragments in shared memory
    static constexpr int kQ = kQShared ? DP / 16 * NT * 32 * 8 : 0;
    static constexpr int kWarpBytes = kStages * kStage + kQ + DP * 4;  // and first tokens whose values are NaN, by entry
    // Warps of a CTA and CTAs of an SM, as registers and shared memory allow: O alone takes DP NT / 4 registers.
    static constexpr int kWarps = DP * NT == 128 ? 8 : DP * NT == 256 ? 12 : 8;
    static constexpr int kCtas = DP * NT == 128 ? 2 : 1;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kBytes = kWarps * kWarpBytes;
};

// The rows [row0, row0 + 8 NT) of sequence s and kv head h over its own tokens [from, to).
template <int DP, int NT>
__device__ __forceinline__ void run_chunk(const ChunkParams &p, const SharedSeq &s, int h, int row0, int from,
                                          int to, float *part, uint8_t *ring, uint2 *sq, int *nan_from) {
    constexpr int kHalves = DP / 128, kSteps = DP / 16, kStages = Chunk<DP, NT>::kStages, kStage = Chunk<DP, NT>::kStage;
    constexpr bool kQShared = NT > 1;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rows = s.q_len * p.g, d = p.c.d;
    const int start = s.kv_len - s.q_len;
    const int *const pages = p.n.table + (size_t)s.row * p.n.table_stride + s.page0;

    // ---- pages of the next 32 steps, a lane each: where the step's codes begin (-1: reads as zeros) and its scales
    long long offset = -1;
    float kscale = 1.f, vlog = 0.f;
    auto page_at = [&](int tok) {
        tok += lane * kStep;
        return tok < to ? pages[tok >> p.c.page_log2] : 0;
    };
    auto look_up = [&](int tok, int page) {
        tok += lane * kStep;
        offset = -1;
        kscale = 1.f;
        vlog = 0.f;
        if (tok < to) {
            if (page < 0 || page >= p.c.pages) {
                atomicOr(p.err, kDevErrAttnInput);
            } else {
                offset = page * p.c.ps + h * p.c.hs + (tok & (p.c.page - 1)) * p.c.ts;
                kscale = p.c.ks[(size_t)page * p.c.heads + h];
                vlog = log2f(p.c.vs[(size_t)page * p.c.heads + h]);
            }
        }
    };
    const int page = page_at(from);
    // ---- the query rows' bf16 pairs, on their way while pages and scales are looked up
    uint32_t u[NT][kSteps][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = row0 + 8 * n + g;
        const bool on = r < rows;
        const int i = on ? p.g_div(r) : 0, hq = h * p.g + (on ? r - i * p.g : 0);
        const uint16_t *const src = p.q.p + (s.t0 + i) * p.q.ts + hq * p.q.hs;
#pragma unroll
        for (int k = 0; k < kSteps; k += 4) {  // 16 entries of this lane
            const int e = k * 16 + 16 * t;
            uint4 a = make_uint4(0, 0, 0, 0), b = a;
            if (on && e < d) {
                a = load_rows8(src + e, p.q.vec);
                b = load_rows8(src + e + 8, p.q.vec);
            }
            u[n][k][0] = a.x, u[n][k][1] = a.y, u[n][k + 1][0] = a.z, u[n][k + 1][1] = a.w;
            u[n][k + 2][0] = b.x, u[n][k + 2][1] = b.y, u[n][k + 3][0] = b.z, u[n][k + 3][1] = b.w;
        }
    }
    look_up(from, page);
    // A step's codes on their way into shared memory: each lane copies what it will read itself, so that nothing but its
    // own copies is waited for, and a warp's reads are 512 contiguous bytes.
    const uint32_t mine = smem_u32(ring) + lane * 16;
    int left = 32;     // steps that the lanes have looked up
    int asked = from;  // the first token that is not asked for
    int slot = 0;      // of the ring, for the next step
    float ks_ahead[kStages], lvs_ahead[kStages];  // scales of the steps asked for, the next one first
    // where a lane's entries lie in a step, and which of them are there
    const long long k_lane = g * p.c.ts + (16 * t < d ? 16 * t : 0), v_lane = 2 * t * p.c.ts + (16 * g < d ? 16 * g : 0);
    int k_size[2 * kHalves], v_size[kHalves];
#pragma unroll
    for (int i = 0; i < 2 * kHalves; ++i) k_size[i] = i * 64 + 16 * t < d ? 16 : 0;
#pragma unroll
    for (int i = 0; i < kHalves; ++i) v_size[i] = i * 128 + 16 * g < d ? 16 : 0;
    auto ask = [&](int n) {  // n: steps ahead of the one that is worked on
        if (asked < to) {
            const int now = 32 - left;
            const long long at = __shfl_sync(0xffffffffu, offset, now);
            ks_ahead[n] = __shfl_sync(0xffffffffu, kscale, now);
            lvs_ahead[n] = __shfl_sync(0xffffffffu, vlog, now);
            const uint32_t to_slot = mine + slot * kStage;
            if (at >= 0) {
                const uint8_t *const k = p.c.k + at + k_lane, *const v = p.c.v + at + v_lane;
#pragma unroll
                for (int i = 0; i < 2 * kHalves; ++i) {
                    copy16(to_slot + (2 * i) * 512, k + (k_size[i] ? i * 64 : 0), k_size[i]);
                    copy16(to_slot + (2 * i + 1) * 512, k + 8 * p.c.ts + (k_size[i] ? i * 64 : 0), k_size[i]);
                }
#pragma unroll
                for (int i = 0; i < kHalves; ++i)
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        copy16(to_slot + (4 * kHalves + 4 * i + z) * 512,
                               v + ((z & 1) + (z >> 1) * 8) * p.c.ts + (v_size[i] ? i * 128 : 0), v_size[i]);
            } else {
#pragma unroll 1
                for (int i = 0; i < 8 * kHalves; ++i) copy16(to_slot + i * 512, p.c.k, 0);
            }
            asked += kStep;
            if (++slot == kStages) slot = 0;
            if (--left == 0) {
                left = 32;
                look_up(asked, page_at(asked));
            }
        }
        copies_commit();
    };
#pragma unroll
    for (int n = 0; n + 1 < kStages; ++n) ask(n);

    // ---- the query rows as B fragments, each scaled by a power of two to a maximum in [2^7, 2^8)
    uint2 qf[kQShared ? 1 : kSteps];
    float qs[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        uint32_t two = 0;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) two = __vmaxu2(two, __vmaxu2(u[n][k][0] & 0x7FFF7FFFu, u[n][k][1] & 0x7FFF7FFFu));
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
            uint32_t f[2];
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const __half2 x = __floats2half2_rn(__uint_as_float(u[n][k][w] << 16) * down,
                                                    __uint_as_float(u[n][k][w] & 0xFFFF0000u) * down);
                f[w] = *reinterpret_cast<const uint32_t *>(&x);
            }
            if constexpr (kQShared)
                sq[(k * NT + n) * 32 + lane] = make_uint2(f[0], f[1]);
            else
                qf[k] = make_uint2(f[0], f[1]);
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

    int read = 0;  // the ring's slot of this step
    for (int tok = from; tok < to; tok += kStep) {
        ask(kStages - 1);
        copies_wait<kStages - 1>();
        const float ks = ks_ahead[0], lvs = lvs_ahead[0];
#pragma unroll
        for (int n = 0; n + 1 < kStages; ++n) {
            ks_ahead[n] = ks_ahead[n + 1];
            lvs_ahead[n] = lvs_ahead[n + 1];
        }
        const uint8_t *const here = ring + read * kStage + lane * 16;
        if (++read == kStages) read = 0;
        auto piece = [&](int i) { return *reinterpret_cast<const uint4 *>(here + i * 512); };
        // ---- scores
        float s0[NT][4], s1[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) s0[n][c] = s1[n][c] = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * kHalves; ++i) {
            const uint4 k0 = piece(2 * i), k1 = piece(2 * i + 1);
            const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
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
#pragma unroll
        for (int i = 0; i < kHalves; ++i) {
            uint4 vf[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) vf[z] = piece(4 * kHalves + 4 * i + z);
            if (edge) {
                // A zero weight does not hide a NaN: codes that nobody sees become zeros, a NaN that only some rows
                // see is noted by entry and token (rows see all tokens from one on).
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const int at = tok + 2 * t + (z & 1) + (z >> 1) * 8;
                    uint32_t *const w = reinterpret_cast<uint32_t *>(&vf[z]);
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
            const uint32_t va[4] = {vf[0].x, vf[0].y, vf[0].z, vf[0].w}, vb[4] = {vf[1].x, vf[1].y, vf[1].z, vf[1].w};
            const uint32_t vc[4] = {vf[2].x, vf[2].y, vf[2].z, vf[2].w}, vd[4] = {vf[3].x, vf[3].y, vf[3].z, vf[3].w};
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
    while (n > 128) {  // [lo, lo + n)
        const int step = (n + 31) / 32, at = lane * step;
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, at < n && __ldcg(sums + lo + min(at, n - 1)) <= x));
        lo += last * step;
        n = min(step, n - last * step);
    }
    int below = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int at = lane + 32 * k;
        below += __popc(__ballot_sync(0xffffffffu, at < n && __ldcg(sums + lo + min(at, n - 1)) <= x));
    }
    return lo + below - 1;
}

// Warps take the next item that nobody has taken: the kernel starts beside the
// prompt kernel, on the SMs that that one leaves, and its other CTAs come as the
// prompt kernel's go, when there may be nothing left.
template <int DP, int NT>
__global__ void __launch_bounds__(Chunk<DP, NT>::kThreads, Chunk<DP, NT>::kCtas) attn_chunks_kernel(const ChunkParams p) {
    using T = Chunk<DP, NT>;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *const ring = smem + warp * T::kWarpBytes;
    uint2 *const sq = reinterpret_cast<uint2 *>(ring + T::kStages * T::kStage);
    int *const nan_from = reinterpret_cast<int *>(ring + T::kStages * T::kStage + T::kQ);
    if (threadIdx.x == 0) griddep_launch_dependents();  // (the join waits for this kernel's end)
    // What follows reads the plan's records, the table, scales, codes and queries ahead of this kernel's own wait.  It may, as
    // this kernel starts only after every CTA of the one ahead (attn_prompt_kernel<.., SharedParams>) has let it, which each
    // does behind its own wait for the plan, and the plan begins with a wait for what was before the call.
    for (int e = lane; e < DP; e += 32) nan_from[e] = 0x7FFFFFFF;
    __syncwarp();
    const int4 head = __ldcg(reinterpret_cast<const int4 *>(p.head));
    const int items = head.x, size = head.y, taken = head.z;
    // Warps of the CTAs that find an SM at once, which begin with an item of their own.
    const int early = (p.ctas - head.w) * T::kCtas * T::kWarps, number = blockIdx.x * T::kWarps + warp;
    auto take = [&] { return lane == 0 ? early + atomicAdd(&p.head->next, 1) : 0; };
    int mine = number;
    if (number >= early) {
        // A later one takes about twice as long for its first item, most of it to fetch its instructions: it helps only
        // where the others would take two more each.
        mine = items - early - taken > early ? take() : items;
    }
    for (;;) {
        const int item = __shfl_sync(0xffffffffu, mine, 0);
        if (item >= items) break;
        const int record = owner_of(p.first, p.n.b, item);
        const int4 *const at = reinterpret_cast<const int4 *>(p.own + record);
        const int4 a = __ldcg(at), b = __ldcg(at + 1);
        SharedSeq s;
        s.t0 = a.x, s.q_len = a.y, s.kv_len = a.z, s.row = a.w;
        s.page0 = b.x, s.chunks = b.z, s.first_item = b.w;
        s.parts = __ldcg(&p.own[record].parts);
        mine = take();
        if (s.chunks == 0) continue;  // passed over
        // numbered by kv head, chunk and block of rows
        const int blocks = (s.q_len * p.g + 8 * NT - 1) / (8 * NT), i = item - s.first_item;
        const int c = i / blocks, row0 = (i - c * blocks) * 8 * NT, h = c / s.chunks, chunk = c - h * s.chunks;
        const int from = chunk * size, to = min(s.kv_len, from + size);
        if (!nvfp4_in_bounds(from < to && h < p.c.heads && s.parts >= 0 &&
                                 (long long)s.parts + (long long)s.chunks * s.q_len * p.g * p.c.heads <= p.room,
                             p.err))
            continue;
        float *const part = p.parts + (s.parts + (long long)c * (s.q_len * p.g)) * (p.c.d + 4);
        run_chunk<DP, NT>(p, s, h, row0, from, to, part, ring, sq, nan_from);
        copies_wait<0>();  // (all have landed; empty groups may be left)
    }
    griddep_wait();  // who waits for this kernel's end waits for the prompt kernel's too
}

template <int DP, int NT>
cudaError_t chunks_launch(const ChunkParams &p, cudaStream_t stream) {
    using T = Chunk<DP, NT>;
    return launch_behind(attn_chunks_kernel<DP, NT>, dim3((unsigned)(p.ctas * T::kCtas)), T::kThreads, (size_t)T::kBytes, stream,
                         p);
}
template <int DP, int NT>
cudaError_t chunks_limit() {
    static_assert(Chunk<DP, NT>::kBytes * Chunk<DP, NT>::kCtas <= 224 * 1024, "shared memory");
    return cudaFuncSetAttribute(attn_chunks_kernel<DP, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Chunk<DP, NT>::kBytes);
}

}  // namespace

cudaError_t attn_chunks_set_smem_limit() {
    cudaError_t e = chunks_limit<128, 1>();
    if (e == cudaSuccess) e = chunks_limit<128, 2>();
    if (e == cudaSuccess) e = chunks_limit<256, 1>();
    return e == cudaSuccess ? chunks_limit<256, 2>() : e;
}

int attn_chunk_warps(int d, bool eight) {
    auto of = [](auto x) { return decltype(x)::kWarps * decltype(x)::kCtas; };
    if (d > 128) return eight ? of(Chunk<256, 1>()) : of(Chunk<256, 2>());
    return eight ? of(Chunk<128, 1>()) : of(Chunk<128, 2>());
}

cudaError_t launch_attn_chunks(const ChunkParams &p, cudaStream_t stream) {
    const bool eight = attn_chunk_rows(p.n.max_q * p.g) == 8;
    if (p.c.d > 128) return eight ? chunks_launch<256, 1>(p, stream) : chunks_launch<256, 2>(p, stream);
    return eight ? chunks_launch<128, 1>(p, stream) : chunks_launch<128, 2>(p, stream);
}

}  // namespace nvfp4
