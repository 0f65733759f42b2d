// attn_heads.cu -- per-head RMS norm and position rotation of queries and
// keys, alone (bf16 to bf16) and on the way into the paged 8-bit cache.
//
// A head of D <= 256 entries is held by a group of L = 8, 16 or 32 lanes,
// eight consecutive entries a lane, so that one 16-byte load a lane reads it:
//
//     y[d] = x[d] * w[d] / sqrt(mean(x^2) + eps)          (fp32)
//     (a, b) -> (a cos - b sin, b cos + a sin)            (fp32, one rounding at the end)
//
// The sum of squares is a shuffle reduction over the group.  Of the pair
// (x[i], x[i + rot / 2]) the other entry lies rot / 16 lanes away when rot / 2
// is a multiple of 8 (four shuffles of packed bf16 pairs); for other rot it is
// loaded again, one entry at a time, from the line just read.  Adjacent pairs
// lie in one lane.
#include "attn.cuh"

namespace nvfp4 {

namespace {

constexpr int kHeadThreads = 256;

__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
// Entries [8 lane, 8 lane + 8) of a head (zeros past D).
__device__ __forceinline__ uint4 load8(const uint16_t *p, int e0, int D, int vec) {
    if (e0 >= D) return make_uint4(0, 0, 0, 0);
    if (vec) return *reinterpret_cast<const uint4 *>(p + e0);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)p[e0 + 2 * i] | ((uint32_t)p[e0 + 2 * i + 1] << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One head, normalised and rotated, by a group of L lanes.  `p`: its D bf16
// entries, `w`: the norm's weight (nullptr: none), `cs`: the position's row of
// the table (nullptr: no rotation).
template <int L>
__device__ __forceinline__ void head8(const uint16_t *p, int vec, const uint16_t *w, const float *cs,
                                      const NormRope &how, int D, int lane, unsigned mask, float (&y)[8]) {
    const int e0 = lane * 8;
    const uint4 raw = load8(p, e0, D, vec);
    unpack8(raw, y);
    float rinv = 1.f;
    if (w) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o, L);
        rinv = __frsqrt_rn(ss / (float)D + how.eps);
        float wf[8];
        unpack8(load8(w, e0, D, 0), wf);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] * rinv * wf[i];
    }
    if (!cs) return;
    const int rot = how.rot, half = rot >> 1;
    if (how.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = e0 + 2 * i;
            if (e < rot) {
                const float c = cs[e >> 1], s = cs[half + (e >> 1)], a = y[2 * i], b = y[2 * i + 1];
                y[2 * i] = fmaf(a, c, -(b * s));
                y[2 * i + 1] = fmaf(b, c, a * s);
            }
        }
        return;
    }
    float other[8];
    if ((half & 7) == 0) {
        // the other half of the pairs lies half / 8 lanes away
        const int src = e0 < half ? lane + (half >> 3) : lane - (half >> 3);
        uint4 o;
        o.x = __shfl_sync(mask, raw.x, src, L);
        o.y = __shfl_sync(mask, raw.y, src, L);
        o.z = __shfl_sync(mask, raw.z, src, L);
        o.w = __shfl_sync(mask, raw.w, src, L);
        unpack8(o, other);
        if (w && e0 < rot) {
            float wf[8];
            unpack8(load8(w, src * 8, D, 0), wf);
#pragma unroll
            for (int i = 0; i < 8; ++i) other[i] = other[i] * rinv * wf[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = e0 + i;
            const int o = e < half ? e + half : e - half;
            other[i] = e < rot ? bf16_f32(p[o]) : 0.f;
            if (w && e < rot) other[i] = other[i] * rinv * bf16_f32(w[o]);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = e0 + i;
        if (e < rot) {
            const int f = e < half ? e : e - half;
            const float c = cs[f], s = cs[half + f];
            y[i] = e < half ? fmaf(y[i], c, -(other[i] * s)) : fmaf(y[i], c, other[i] * s);
        }
    }
}

__device__ __forceinline__ void store8(uint16_t *p, const float (&y)[8], int e0, int D) {
    if (e0 < D)
        *reinterpret_cast<uint4 *>(p + e0) =
            make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
}

// ------------------------------------------------------------- norm + rotation
// One group of L lanes for every (token, head), the query heads of a token
// before its key heads.
template <int L>
__global__ void __launch_bounds__(kHeadThreads)
    norm_rope_kernel(HeadRows q, HeadRows k, const int *__restrict__ positions, NormRope how, int tokens, int D,
                     uint16_t *q_out, uint16_t *k_out, unsigned *err) {
    constexpr int kGroups = kHeadThreads / L;
    const int lane = threadIdx.x % L;
    const unsigned mask = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << ((threadIdx.x & 31) / L * L);
    const int heads = q.heads + k.heads;
    const long long unit = (long long)blockIdx.x * kGroups + threadIdx.x / L;
    if (unit >= (long long)tokens * heads) return;
    const int t = (int)(unit / heads), h = (int)(unit - (long long)t * heads);
    const bool is_k = h >= q.heads;
    const int hh = is_k ? h - q.heads : h;
    const HeadRows &r = is_k ? k : q;
    float y[8];
    const float *cs = nullptr;
    bool ok = true;
    if (how.rot > 0) {
        const int pos = positions[t];
        ok = pos >= 0 && pos < how.positions;
        if (!ok && lane == 0) atomicOr(err, kDevErrAttnInput);
        cs = how.cs + (size_t)(ok ? pos : 0) * how.rot;
    }
    head8<L>(r.p + t * r.ts + hh * r.hs, r.vec, is_k ? how.kw : how.qw, cs, how, D, lane, mask, y);
    if (!ok) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = 0.f;
    }
    store8((is_k ? k_out : q_out) + ((size_t)t * r.heads + hh) * D, y, lane * 8, D);
}

// ---------------------------------------------------------------------- append
struct AppendParams {
    HeadRows q, k, v;
    NormRope how;
    KvCache c;
    KvBatch n;
    uint16_t *q_out;
    unsigned *err;
    int page_span;  // pages that max_q_len tokens can touch
    int roles;      // key heads, value heads, query heads
};

// The smallest power of two s with amax <= 448 s, within 2^-100 .. 2^100.
__device__ __forceinline__ float need_scale(float amax) {
    if (!(amax > 0.f)) return __int_as_float((127 - 100) << 23);
    const uint32_t u = __float_as_uint(amax);
    int e = (int)(u >> 23) - 127 - 8;               // amax = 1.m 2^(e + 8); 448 = 1.75 2^8
    if ((u & 0x7FFFFFu) > 0x600000u) ++e;            // 1.m > 1.75
    e = min(max(e, -100), 100);                      // an fp32 subnormal has e = -135 here
    return __int_as_float((127 + e) << 23);
}

// x / s, with the product by the exact reciprocal where s is a power of two.
struct Divisor {
    float s, inv;
    bool pow2;
    __device__ explicit Divisor(float v) {
        s = v;
        inv = 1.f / v;
        pow2 = (__float_as_uint(v) & 0x7FFFFFu) == 0u;
    }
    __device__ float operator()(float x) const { return pow2 ? x * inv : __fdiv_rn(x, s); }
};

// Four values -> four E4M3 codes (nearest, ties to even, saturated; an
// infinity or NaN becomes NaN).
__device__ __forceinline__ float finite_or_nan(float x) { return x - x == 0.f ? x : __int_as_float(0x7FC00000); }
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n .reg .b16 lo, hi;\n"
        " cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
        " mov.b32 %0, {lo, hi};\n}\n"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
__device__ __forceinline__ void e4m3x4_f32(uint32_t v, float (&x)[4]) {
    const uint32_t a = e4m3x2_to_f16x2(v), b = e4m3x2_to_f16x2(v >> 16);
    const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&a));
    const float2 q = __half22float2(*reinterpret_cast<const __half2 *>(&b));
    x[0] = p.x;
    x[1] = p.y;
    x[2] = q.x;
    x[3] = q.y;
}

// A unit is (sequence, one of the pages its new tokens touch, role), a role a
// key head, a value head or a query head.  kBlock: a CTA takes a unit, its
// groups the page's tokens side by side (prompts).  Otherwise a single group
// takes it, one token after the other (a few tokens a sequence: decode).
template <int L, bool kBlock>
__global__ void __launch_bounds__(kHeadThreads) kv_append_kernel(const AppendParams p) {
    constexpr int kGroups = kHeadThreads / L;
    const int group = threadIdx.x / L, lane = threadIdx.x % L, e0 = lane * 8;
    const unsigned mask = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << ((threadIdx.x & 31) / L * L);
    const long long unit = kBlock ? (long long)blockIdx.x : (long long)blockIdx.x * kGroups + group;
    if (unit >= (long long)p.n.b * p.page_span * p.roles) return;
    const int D = p.c.d, first = kBlock ? group : 0, step = kBlock ? kGroups : 1;
    const int role = (int)(unit % p.roles);
    const int bj = (int)(unit / p.roles), b = bj / p.page_span, j = bj - b * p.page_span;
    int t0, q_len, kv_len;
    if (!kv_sequence(p.n, b, &t0, &q_len, &kv_len) && lane == 0) atomicOr(p.err, kDevErrAttnInput);
    const int start = kv_len - q_len;  // position of the sequence's first new token
    const bool is_q = role >= 2 * p.c.heads, is_v = !is_q && role >= p.c.heads;
    const int h = is_q ? role - 2 * p.c.heads : is_v ? role - p.c.heads : role;
    const HeadRows &rows = is_q ? p.q : is_v ? p.v : p.k;
    const uint16_t *src = rows.p + h * rows.hs;
    const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (is_q && j == 0)  // tokens without a place in the sequence
        for (int pos = start + first; pos < 0; pos += step)
            store8(p.q_out + ((size_t)(t0 + pos - start) * p.q.heads + h) * D, zero, e0, D);
    const int pg = (max(start, 0) >> p.c.page_log2) + j, base = pg << p.c.page_log2;
    const int lo = max(max(start, 0), base), hi = min(kv_len, base + p.c.page);
    if (lo >= hi) return;
    const uint16_t *w = is_v ? nullptr : is_q ? p.how.qw : p.how.kw;
    auto value = [&](int pos, float (&x)[8]) {
        const float *cs = is_v || p.how.rot == 0 ? nullptr : p.how.cs + (size_t)pos * p.how.rot;
        head8<L>(src + (t0 + pos - start) * rows.ts, rows.vec, w, cs, p.how, D, lane, mask, x);
    };
    float x[8];
    if (is_q) {
        for (int pos = lo + first; pos < hi; pos += step) {
            value(pos, x);
            store8(p.q_out + ((size_t)(t0 + pos - start) * p.q.heads + h) * D, x, e0, D);
        }
        return;
    }
    const int page = p.n.table[(size_t)b * p.n.table_stride + pg];
    if (page < 0 || page >= p.c.pages) {
        if (lane == 0) atomicOr(p.err, kDevErrAttnInput);
        return;
    }
    float amax = 0.f;
    for (int pos = lo + first; pos < hi; pos += step) {
        value(pos, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = x[i] - x[i] == 0.f ? fmaxf(amax, fabsf(x[i])) : amax;
    }
    float *const sp = (is_v ? p.c.vs : p.c.ks) + (size_t)page * p.c.heads + h;
    const float old = lo > base ? *sp : 0.f;  // read before the barrier, written after it
    if (kBlock) {
        __shared__ float part[kHeadThreads / 32];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kHeadThreads / 32; ++i) amax = fmaxf(amax, part[i]);
    } else {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(mask, amax, o, L));
    }
    const float s = fmaxf(need_scale(amax), old);
    uint8_t *const codes = (is_v ? p.c.v : p.c.k) + (size_t)page * p.c.ps + (size_t)h * p.c.hs + e0;
    if (first == 0 && lane == 0) *sp = s;
    if (s > old && lo > base && e0 < D) {  // the page's earlier tokens, for the larger scale
        const float ratio = old / s;
        for (int slot = first; slot < lo - base; slot += step) {
            uint2 *const c = reinterpret_cast<uint2 *>(codes + (size_t)slot * p.c.ts);
            uint2 v = *c;
            float a[4], d[4];
            e4m3x4_f32(v.x, a);
            e4m3x4_f32(v.y, d);
            v.x = e4m3x4(a[0] * ratio, a[1] * ratio, a[2] * ratio, a[3] * ratio);
            v.y = e4m3x4(d[0] * ratio, d[1] * ratio, d[2] * ratio, d[3] * ratio);
            *c = v;
        }
    }
    const Divisor div(s);
    for (int pos = lo + first; pos < hi; pos += step) {
        if (hi - lo > step) value(pos, x);  // else the only one, still held
        float z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = finite_or_nan(div(x[i]));
        if (e0 < D)
            *reinterpret_cast<uint2 *>(codes + (size_t)(pos - base) * p.c.ts) =
                make_uint2(e4m3x4(z[0], z[1], z[2], z[3]), e4m3x4(z[4], z[5], z[6], z[7]));
    }
}

template <int L>
cudaError_t append_l(const AppendParams &p, cudaStream_t stream) {
    const long long units = (long long)p.n.b * p.page_span * p.roles;
    // A group a unit while a unit is at most two tokens; a CTA a unit above.
    if (p.n.max_q <= 2) {
        constexpr int kGroups = kHeadThreads / L;
        kv_append_kernel<L, false><<<(unsigned)((units + kGroups - 1) / kGroups), kHeadThreads, 0, stream>>>(p);
    } else {
        kv_append_kernel<L, true><<<(unsigned)units, kHeadThreads, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const HeadRows &q, const HeadRows &k, const int *positions, const NormRope &how,
                             int tokens, int d, uint16_t *q_out, uint16_t *k_out, unsigned *err,
                             cudaStream_t stream) {
    const long long heads = (long long)tokens * (q.heads + k.heads);
    const int L = d > 128 ? 32 : d > 64 ? 16 : 8;
    const unsigned grid = (unsigned)((heads * L + kHeadThreads - 1) / kHeadThreads);
    if (L == 32)
        norm_rope_kernel<32><<<grid, kHeadThreads, 0, stream>>>(q, k, positions, how, tokens, d, q_out, k_out, err);
    else if (L == 16)
        norm_rope_kernel<16><<<grid, kHeadThreads, 0, stream>>>(q, k, positions, how, tokens, d, q_out, k_out, err);
    else
        norm_rope_kernel<8><<<grid, kHeadThreads, 0, stream>>>(q, k, positions, how, tokens, d, q_out, k_out, err);
    return cudaGetLastError();
}

cudaError_t launch_kv_append(const HeadRows &q, const HeadRows &k, const HeadRows &v, const NormRope &how,
                             const KvCache &c, const KvBatch &n, uint16_t *q_out, unsigned *err,
                             cudaStream_t stream) {
    AppendParams p;
    p.q = q;
    p.k = k;
    p.v = v;
    p.how = how;
    p.c = c;
    p.n = n;
    p.q_out = q_out;
    p.err = err;
    p.page_span = (n.max_q + c.page - 2) / c.page + 1;
    p.roles = 2 * c.heads + q.heads;
    return c.d > 128 ? append_l<32>(p, stream) : c.d > 64 ? append_l<16>(p, stream) : append_l<8>(p, stream);
}

}  // namespace nvfp4
