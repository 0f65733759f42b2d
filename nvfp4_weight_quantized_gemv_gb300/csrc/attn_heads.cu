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
//
// Both kernels move bytes and little else, but 8-entry lanes give an SM's
// schedulers about as much to issue as HBM takes: 135 instructions a head of 256
// for the norm and rotation, 155 for the append (of which the rotation's table
// and weights are shared by the heads of a token).  So a group requests several
// heads (or tokens) before it works on the first, and the paths for pairs and
// alignments are kernels of their own: one kernel with branches took 70 us
// where these take 46.
// 8192 tokens of 24 + 4 heads of 256: norm and rotation 237 MB in 46 us, 5.1
// TB/s (0.76 of a plain copy's rate); append (24 + 4 + 4 heads into pages of 64)
// 254 MB in 61 us, 4.1 TB/s.  A token alone 1.9 us, 16 sequences of one token
// appended 3.4 us: a launch and three dependent loads.
#include "attn.cuh"

#include <type_traits>

namespace nvfp4 {

namespace {

constexpr int kHeadThreads = 256;
constexpr int kNormCtas = 3;  // an SM's, at 80 registers; four at 64 spill and take as long

// Eight bf16 -> fp32.
__device__ __forceinline__ void unpack8(const uint4 &v, float2 (&x)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ void store8(uint16_t *p, const float2 (&y)[4]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(y[0].x, y[0].y), pack_bf16(y[1].x, y[1].y),
                                               pack_bf16(y[2].x, y[2].y), pack_bf16(y[3].x, y[3].y));
}
__device__ __forceinline__ uint32_t swap16(uint32_t v) { return __byte_perm(v, v, 0x1032); }

// How the entries of a rotated pair lie, and how they can be loaded: a fixed
// half apart, a whole number of lanes; side by side; anything, by halves that
// are no whole number of lanes or in memory without the alignment for 16-byte
// loads (of heads, weights and table alike).
enum Pairs { kHalves, kAdjacent, kAny };

template <int kPairs>
__device__ __forceinline__ uint4 load_head8(const uint16_t *p, int vec) {
    return load_rows8(p, kPairs != kAny || vec);
}

// A lane's place in its group, with the norm's weights (bf16) of its entries
// and of those that they are paired with, the latter with the sign of the
// pair's second product, zero where an entry has no partner.  Norm and
// rotation are then, whatever the pairing,
//
//     y[e] = (x[e] (w[e] cos) + x[other(e)] (+-w[other(e)] sin)) / rms,
//
// with a rounding of fp32 at w cos and w sin, which the heads of a token share,
// where x w / rms would have one: in the append of 8192 tokens 3 to 6 of 8.4 million
// keys' E4M3 codes are the neighbours of exact arithmetic's (5 to 8 the other way).
template <int L, int kPairs>
struct Lane {
    int lane, e0;
    unsigned mask;
    bool on, norm;
    bool side;  // pairs side by side
    bool far;   // half-split pairs that are not a whole number of lanes apart
    int from;  // the lane with the partners, of a half-split that is not far
    uint4 w, wo;
    __device__ __forceinline__ Lane(const NormRope &how, const uint16_t *weight, int w_vec, int D) {
        lane = threadIdx.x % L;
        e0 = lane * 8;
        mask = L == 32 ? 0xffffffffu : ((1u << L) - 1u) << ((threadIdx.x & 31) / L * L);
        on = e0 < D;
        norm = weight != nullptr;
        const int half = how.rot >> 1;
        side = kPairs == kAny ? how.interleaved != 0 : kPairs == kAdjacent;
        far = kPairs == kAny && !side && (half & 7) != 0;
        const bool paired = !side && !far && e0 < how.rot;
        from = !paired ? lane : e0 < half ? lane + (half >> 3) : lane - (half >> 3);
        const uint4 ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
        w = !norm ? ones : on ? load_head8<kPairs>(weight + e0, w_vec) : make_uint4(0, 0, 0, 0);
        wo = make_uint4(0, 0, 0, 0);
        if (side) {
            wo.x = e0 < how.rot ? swap16(w.x) ^ 0x8000u : 0u;
            wo.y = e0 + 2 < how.rot ? swap16(w.y) ^ 0x8000u : 0u;
            wo.z = e0 + 4 < how.rot ? swap16(w.z) ^ 0x8000u : 0u;
            wo.w = e0 + 6 < how.rot ? swap16(w.w) ^ 0x8000u : 0u;
        } else if (paired) {
            wo = norm ? load_head8<kPairs>(weight + from * 8, w_vec) : ones;
            const uint32_t sign = e0 < half ? 0x80008000u : 0u;
            wo.x ^= sign, wo.y ^= sign, wo.z ^= sign, wo.w ^= sign;
        } else if (far) {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = e0 + i;
                v[i] = e >= how.rot ? 0u : norm ? weight[e < half ? e + half : e - half] : 0x3F80u;
                if (e < half) v[i] ^= 0x8000u;
            }
            wo = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
        }
    }
};

// The two factors of each entry at a position: w cos and +-w[other] sin.
struct Turn {
    float2 own[4], other[4];
};
template <int L, int kPairs>
__device__ __forceinline__ void make_turn(const Lane<L, kPairs> &ln, const NormRope &how, int pos, Turn &t) {
    unpack8(ln.w, t.own);
    if (how.rot == 0) return;
    unpack8(ln.wo, t.other);
    if (ln.e0 >= how.rot) return;
    const float *const cs = how.cs + (size_t)pos * how.rot;
    const int half = how.rot >> 1;
    const bool vec = kPairs != kAny || how.cs_vec;
    if (ln.side) {
        const int f = ln.e0 >> 1;
        float c[4], s[4];
        if (vec) {
            const float4 cv = *reinterpret_cast<const float4 *>(cs + f);
            const float4 sv = *reinterpret_cast<const float4 *>(cs + half + f);
            c[0] = cv.x, c[1] = cv.y, c[2] = cv.z, c[3] = cv.w;
            s[0] = sv.x, s[1] = sv.y, s[2] = sv.z, s[3] = sv.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = f + i < half ? cs[f + i] : 1.f;
                s[i] = f + i < half ? cs[half + f + i] : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t.own[i] = mul2(t.own[i], make_float2(c[i], c[i]));
            t.other[i] = mul2(t.other[i], make_float2(s[i], s[i]));
        }
        return;
    }
    float2 c[4], s[4];
    if (vec && !ln.far) {
        const float *const at = cs + (ln.e0 < half ? ln.e0 : ln.e0 - half);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 cv = *reinterpret_cast<const float4 *>(at + 4 * i);
            const float4 sv = *reinterpret_cast<const float4 *>(at + half + 4 * i);
            c[2 * i] = make_float2(cv.x, cv.y), c[2 * i + 1] = make_float2(cv.z, cv.w);
            s[2 * i] = make_float2(sv.x, sv.y), s[2 * i + 1] = make_float2(sv.z, sv.w);
        }
    } else {
        float cc[8], ss[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = ln.e0 + i, f = e < half ? e : e - half;
            cc[i] = e < how.rot ? cs[f] : 1.f;
            ss[i] = e < how.rot ? cs[half + f] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = make_float2(cc[2 * i], cc[2 * i + 1]);
            s[i] = make_float2(ss[2 * i], ss[2 * i + 1]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        t.own[i] = mul2(t.own[i], c[i]);
        t.other[i] = mul2(t.other[i], s[i]);
    }
}

// One head: this lane's eight entries (p: the whole head, from which far
// partners are loaded again) -> y.  kFine: 1 / rms correctly rounded (rsqrtf: 2
// ulp), for what becomes E4M3 codes, where an ulp at a boundary is a whole code.
template <bool kFine, int L, int kPairs>
__device__ __forceinline__ void head8(const Lane<L, kPairs> &ln, const NormRope &how, const uint4 &raw, const uint16_t *p,
                                      const Turn &t, float inv_d, float2 (&y)[4]) {
    float2 x[4];
    unpack8(raw, x);
    float r = 1.f;
    if (ln.norm) {
        float2 s2 = mul2(x[0], x[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) s2 = fma2(x[i], x[i], s2);
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(ln.mask, ss, o, L);
        const float mean = fmaf(ss, inv_d, how.eps);
        r = kFine ? __frsqrt_rn(mean) : rsqrtf(mean);
    }
    const float2 rr = make_float2(r, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = mul2(x[i], t.own[i]);
    if (how.rot == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], rr);
        return;
    }
    uint4 o;
    if (ln.side) {
        o.x = ln.e0 < how.rot ? swap16(raw.x) : 0u;
        o.y = ln.e0 + 2 < how.rot ? swap16(raw.y) : 0u;
        o.z = ln.e0 + 4 < how.rot ? swap16(raw.z) : 0u;
        o.w = ln.e0 + 6 < how.rot ? swap16(raw.w) : 0u;
    } else if (!ln.far) {
        o.x = __shfl_sync(ln.mask, raw.x, ln.from, L);
        o.y = __shfl_sync(ln.mask, raw.y, ln.from, L);
        o.z = __shfl_sync(ln.mask, raw.z, ln.from, L);
        o.w = __shfl_sync(ln.mask, raw.w, ln.from, L);
        if (ln.e0 >= how.rot) o = make_uint4(0, 0, 0, 0);
    } else {
        const int half = how.rot >> 1;
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = ln.e0 + i;
            v[i] = e >= how.rot ? 0u : p[e < half ? e + half : e - half];
        }
        __syncwarp(ln.mask);  // read by all lanes before one stores, should the output be the input's memory
        o = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
    float2 z[4];
    unpack8(o, z);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = mul2(fma2(z[i], t.other[i], y[i]), rr);
}

// ------------------------------------------------------------- norm + rotation
// A group of L lanes takes kHeads consecutive heads of a token, all query
// heads or all key heads: they share the factors of that position.  It does so
// for a few tokens (grid.y), with the same heads (grid.x).
template <int kPairs, int kHeads>
__device__ __forceinline__ void load_heads(uint4 (&raw)[kHeads], const HeadRows &rows, const uint16_t *p, int n, bool on) {
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
        raw[i] = on && i < n ? load_head8<kPairs>(p + i * rows.hs, rows.vec) : make_uint4(0, 0, 0, 0);
}

template <int L, int kPairs, int kHeads>
__global__ void __launch_bounds__(kHeadThreads, kNormCtas)
    norm_rope_kernel(HeadRows q, HeadRows k, const int *positions, NormRope how, int tokens, int rounds, int D,
                     uint16_t *q_out, uint16_t *k_out, unsigned *err) {
    griddep_wait();
    griddep_launch_dependents();
    const int q_sets = (q.heads + kHeads - 1) / kHeads;
    const bool is_k = (int)blockIdx.x >= q_sets;
    const HeadRows &rows = is_k ? k : q;
    const int h0 = (is_k ? (int)blockIdx.x - q_sets : (int)blockIdx.x) * kHeads, n = min(rows.heads - h0, kHeads);
    const Lane<L, kPairs> ln(how, is_k ? how.kw : how.qw, is_k ? how.kw_vec : how.qw_vec, D);
    uint16_t *const dst = (is_k ? k_out : q_out) + h0 * D + ln.e0;
    const float inv_d = 1.f / (float)D;
    constexpr int kStep = kHeadThreads / L;
    const int first = blockIdx.y * (kStep * rounds) + threadIdx.x / L;
    const int last = min(tokens - first, kStep * rounds);
    for (int i = 0; i < last; i += kStep) {
        const int t = first + i;
        const uint16_t *const src = rows.p + t * rows.ts + h0 * rows.hs;
        uint4 raw[kHeads];
        load_heads<kPairs>(raw, rows, src + ln.e0, n, ln.on);
        int pos = 0;
        bool ok = true;
        if (how.rot > 0) {
            pos = positions[t];
            ok = pos >= 0 && pos < how.positions;
            if (!ok && blockIdx.x == 0 && ln.lane == 0) atomicOr(err, kDevErrAttnInput);
        }
        if (!ok) {
            const float2 zero[4] = {};
            for (int i = 0; i < n && ln.on; ++i) store8(dst + ((size_t)t * rows.heads + i) * D, zero);
            continue;
        }
        Turn turn;
        make_turn(ln, how, pos, turn);
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            if (kPairs == kAny && i >= n) break;  // the others go on with zeros: no branch between the heads
            float2 y[4];
            head8<false>(ln, how, raw[i], src + i * rows.hs, turn, inv_d, y);
            if (ln.on && i < n) store8(dst + ((size_t)t * rows.heads + i) * D, y);
        }
    }
}

// ---------------------------------------------------------------------- append
struct AppendParams {
    HeadRows q, k, v;
    NormRope how;
    KvCache c;
    KvBatch n;
    uint16_t *q_out;
    unsigned *err;
    int held;
    unsigned units;
    int page_span;  // pages that max_q_len tokens can touch
    int q_sets, q_parts;  // a page's query heads, kHold a set, and its tokens in as many shares
    int team;             // groups of lanes that work on a unit together
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

// Four values -> four E4M3 codes (nearest, ties to even, saturated; an
// infinity or NaN becomes NaN).
__device__ __forceinline__ float finite_or_nan(float x) { return x - x == 0.f ? x : __int_as_float(0x7FC00000); }
__device__ __forceinline__ uint32_t e4m3x4(float2 a, float2 b) {
    uint32_t r;
    asm("{\n .reg .b16 lo, hi;\n"
        " cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
        " mov.b32 %0, {lo, hi};\n}\n"
        : "=r"(r)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4_times(uint32_t v, float2 ratio) {
    uint32_t a, b;
    e4m3x4_f16(v, a, b);
    return e4m3x4(mul2(__half22float2(*reinterpret_cast<const __half2 *>(&a)), ratio),
                  mul2(__half22float2(*reinterpret_cast<const __half2 *>(&b)), ratio));
}

// A unit is (sequence, one of the pages its new tokens touch, role), a role one
// of: up to kHold query heads of a share of the page's tokens; a key head; a
// value head.  A team of groups takes it, its tokens side by side.  A group
// loads kHold heads of a token together, or of a key or value head kHold
// tokens.  What those become is kept in shared memory, every lane its own
// entries, while the page's scale is settled; where a page is too large for
// that (`held` 0) it is made again.  A team is as large as the page and the
// call's tokens need, up to the whole CTA.
constexpr int kHold = 4;
constexpr int kQTokens = 4;              // query tokens a group takes one after the other (2: 66 us, 8: 64 us for 61)
constexpr int kHeldBytes = 64 * 1024;    // so that three CTAs share an SM (two of more registers, eight tokens
                                         // together: 76 us for 61)

template <int L, int kPairs>
__global__ void __launch_bounds__(kHeadThreads, 3) kv_append_kernel(const AppendParams p) {
    constexpr int kGroups = kHeadThreads / L;
    extern __shared__ __align__(16) float4 held[];
    __shared__ float part[kHeadThreads / 32];
    const int group = threadIdx.x / L, step = p.team, first = group & (step - 1);
    const unsigned unit = blockIdx.x * (unsigned)(kGroups / step) + group / step;
    const unsigned q_roles = p.q_sets * p.q_parts, roles = q_roles + 2 * p.c.heads;
    griddep_wait();
    griddep_launch_dependents();
    if (unit >= p.units) return;
    const int D = p.c.d;
    const unsigned bj = unit / roles;
    const int b = (int)(bj / p.page_span), j = (int)(bj - (unsigned)b * p.page_span);
    unsigned role = unit - bj * roles;
    int t0, q_len, kv_len;
    if (!kv_sequence(p.n, b, &t0, &q_len, &kv_len) && threadIdx.x % L == 0) atomicOr(p.err, kDevErrAttnInput);
    const int start = kv_len - q_len;  // position of the sequence's first new token
    const int pg = (max(start, 0) >> p.c.page_log2) + j, base = pg << p.c.page_log2;
    const int lo = max(max(start, 0), base), hi = min(kv_len, base + p.c.page);
    const float inv_d = 1.f / (float)D;
    Turn turn;

    if (role < q_roles) {
        const int set = (int)(role / (unsigned)p.q_parts), part = (int)role - set * p.q_parts;
        const int h0 = set * kHold, n = min(p.q.heads - h0, kHold);
        const Lane<L, kPairs> ln(p.how, p.how.qw, p.how.qw_vec, D);
        uint16_t *const out = p.q_out + (size_t)h0 * D + ln.e0;
        if (j == 0 && part == 0 && ln.on) {  // tokens without a place in the sequence
            const float2 zero[4] = {};
            for (int pos = start + first; pos < 0; pos += step)
                for (int i = 0; i < n; ++i) store8(out + ((size_t)(t0 + pos - start) * p.q.heads + i) * D, zero);
        }
        for (int pos = lo + part * step + first; pos < hi; pos += p.q_parts * step) {
            const uint16_t *const src = p.q.p + (t0 + pos - start) * p.q.ts + h0 * p.q.hs;
            uint4 raw[kHold];
            load_heads<kPairs>(raw, p.q, src + ln.e0, n, ln.on);
            make_turn(ln, p.how, pos, turn);
#pragma unroll
            for (int i = 0; i < kHold; ++i) {
                if (kPairs == kAny && i >= n) break;
                float2 y[4];
                head8<false>(ln, p.how, raw[i], src + i * p.q.hs, turn, inv_d, y);
                if (ln.on && i < n) store8(out + ((size_t)(t0 + pos - start) * p.q.heads + i) * D, y);
            }
        }
        return;
    }

    role -= q_roles;
    if (lo >= hi) return;  // the whole team, here and below
    const int page = p.n.table[(size_t)b * p.n.table_stride + pg];
    const bool is_v = (int)role >= p.c.heads;
    const int h = is_v ? (int)role - p.c.heads : (int)role;
    const Lane<L, kPairs> ln(p.how, is_v ? nullptr : p.how.kw, p.how.kw_vec, D);
    if (page < 0 || page >= p.c.pages) {
        if (ln.lane == 0) atomicOr(p.err, kDevErrAttnInput);
        return;
    }
    const HeadRows &rows = is_v ? p.v : p.k;
    const uint16_t *const src = rows.p + (t0 - start) * rows.ts + h * rows.hs;
    float *const sp = (is_v ? p.c.vs : p.c.ks) + (size_t)page * p.c.heads + h;
    const float old = lo > base ? *sp : 0.f;  // read before the barrier, written after it
    // One token's entries; infinities become NaN, which no maximum counts.
    auto make = [&](int pos, const uint4 &raw, float2 (&y)[4]) {
        if (is_v) {
            unpack8(raw, y);
        } else {
            make_turn(ln, p.how, pos, turn);
            head8<true>(ln, p.how, raw, src + pos * rows.ts, turn, inv_d, y);
        }
        float most = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) most = fmaxf(most, fmaxf(fabsf(y[e].x), fabsf(y[e].y)));
        if (most > 3.4028235e38f) {
            most = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[e] = make_float2(finite_or_nan(y[e].x), finite_or_nan(y[e].y));
                most = fmaxf(most, fmaxf(fabsf(y[e].x), fabsf(y[e].y)));
            }
        }
        return most;
    };
    float4 *mine = held + threadIdx.x;
    float amax = 0.f;
    for (int from = lo + first; from < hi; from += kHold * step) {
        uint4 raw[kHold];
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            const int pos = from + i * step;
            raw[i] = pos < hi && ln.on ? load_head8<kPairs>(src + pos * rows.ts + ln.e0, rows.vec) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            const int pos = from + i * step;
            if (pos >= hi) break;
            float2 y[4];
            amax = fmaxf(amax, make(pos, raw[i], y));
            if (p.held) {
                mine[0] = make_float4(y[0].x, y[0].y, y[1].x, y[1].y);
                mine[kHeadThreads] = make_float4(y[2].x, y[2].y, y[3].x, y[3].y);
                mine += 2 * kHeadThreads;
            }
        }
    }
    if (step * L > 32) {  // a team of whole warps
        const int warps = step * L / 32, w0 = (threadIdx.x >> 5) & -warps;
        amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));  // not negative
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
        named_barrier(1 + w0 / warps, step * L);
        for (int i = 0; i < warps; ++i) amax = fmaxf(amax, part[w0 + i]);
    } else {
        const unsigned team =
            step * L == 32 ? 0xffffffffu : ((1u << (step * L)) - 1u) << ((threadIdx.x & 31) & -(step * L));
        amax = __uint_as_float(__reduce_max_sync(team, __float_as_uint(amax)));
    }
    const float s = fmaxf(need_scale(amax), old);
    uint8_t *const codes = (is_v ? p.c.v : p.c.k) + (size_t)page * p.c.ps + (size_t)h * p.c.hs + ln.e0;
    if (first == 0 && ln.lane == 0) *sp = s;
    if (s > old && lo > base && ln.on) {  // the page's earlier tokens, for the larger scale
        const float2 ratio = make_float2(old / s, old / s);
        for (int slot = first; slot < lo - base; slot += step) {
            uint2 *const c = reinterpret_cast<uint2 *>(codes + (size_t)slot * p.c.ts);
            const uint2 v = *c;
            *c = make_uint2(e4m3x4_times(v.x, ratio), e4m3x4_times(v.y, ratio));
        }
    }
    // y / s: a product by the exact reciprocal where s is a power of two, as it
    // is unless the caller brought another along.
    const bool pow2 = (__float_as_uint(s) & 0x7FFFFFu) == 0u;
    const float2 inv = make_float2(1.f / s, 1.f / s);
    mine = held + threadIdx.x;
    for (int pos = lo + first; pos < hi; pos += step) {
        float2 y[4];
        if (p.held) {
            const float4 u = mine[0], v = mine[kHeadThreads];
            mine += 2 * kHeadThreads;
            y[0] = make_float2(u.x, u.y), y[1] = make_float2(u.z, u.w);
            y[2] = make_float2(v.x, v.y), y[3] = make_float2(v.z, v.w);
        } else {
            make(pos, ln.on ? load_head8<kPairs>(src + pos * rows.ts + ln.e0, rows.vec) : make_uint4(0, 0, 0, 0), y);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y[e] = pow2 ? mul2(y[e], inv) : make_float2(__fdiv_rn(y[e].x, s), __fdiv_rn(y[e].y, s));
        if (ln.on)
            *reinterpret_cast<uint2 *>(codes + (size_t)(pos - base) * p.c.ts) =
                make_uint2(e4m3x4(y[0], y[1]), e4m3x4(y[2], y[3]));
    }
}

template <int L, int kPairs>
cudaError_t append_l(AppendParams p, cudaStream_t stream) {
    constexpr int kGroups = kHeadThreads / L;
    const int most = p.n.max_q < p.c.page ? p.n.max_q : p.c.page;  // tokens of a unit
    p.team = 1;
    while (p.team < kGroups && p.team * kHold < most) p.team *= 2;
    p.q_sets = (p.q.heads + kHold - 1) / kHold;
    p.q_parts = (most + p.team * kQTokens - 1) / (p.team * kQTokens);
    // A lane's 32 bytes for each of its team's rounds.
    const int bytes = (most + p.team - 1) / p.team * kHeadThreads * 32;
    p.held = bytes <= kHeldBytes;
    const int per = kGroups / p.team;
    const long long units = (long long)p.n.b * p.page_span * (p.q_sets * p.q_parts + 2 * p.c.heads);
    if (units > 0xFFFFFFFFll - per) return cudaErrorInvalidValue;
    p.units = (unsigned)units;
    return launch_behind(kv_append_kernel<L, kPairs>, dim3((p.units + per - 1) / per), kHeadThreads, p.held ? bytes : 0,
                         stream, p);
}

template <int L, int kPairs>
cudaError_t norm_rope_l(const HeadRows &q, const HeadRows &k, const int *positions, const NormRope &how, int tokens,
                        int d, uint16_t *q_out, uint16_t *k_out, unsigned *err, int sms, cudaStream_t stream) {
    constexpr int kGroups = kHeadThreads / L;
    // Four heads a group, of one to eight tokens, where that gives every CTA's slot a unit; else one head of one
    // token.  24 + 4 heads of 256: 256 tokens take 4.3 us with one head and 13 with four, 1024 tokens 12.7
    // and 7.2.
    const int sets = (q.heads + 3) / 4 + (k.heads + 3) / 4;
    const long long each = (long long)sets * tokens / ((long long)kGroups * sms * kNormCtas);
    const bool fill = each > 0;
    const int rounds = max((int)min(max(each, 1LL), 8LL), (tokens / 65535 + kGroups) / kGroups);  // grid.y < 65536
    const int blocks = (int)(((long long)tokens + rounds * kGroups - 1) / (rounds * kGroups));
    return launch_behind(fill ? norm_rope_kernel<L, kPairs, 4> : norm_rope_kernel<L, kPairs, 1>,
                         dim3(fill ? sets : q.heads + k.heads, blocks), kHeadThreads, 0, stream, q, k, positions, how,
                         tokens, rounds, d, q_out, k_out, err);
}

Pairs pairs_of(const NormRope &how, bool rows_vec) {
    if (!rows_vec || !how.qw_vec || !how.kw_vec || (how.rot > 0 && !how.cs_vec)) return kAny;
    return how.interleaved ? kAdjacent : how.rot % 16 == 0 ? kHalves : kAny;
}

// f(L, pairs) with both as constants.
template <int L, class F>
cudaError_t with_pairs(Pairs pairs, F f) {
    using std::integral_constant;
    const integral_constant<int, L> l;
    return pairs == kHalves     ? f(l, integral_constant<int, kHalves>())
           : pairs == kAdjacent ? f(l, integral_constant<int, kAdjacent>())
                                : f(l, integral_constant<int, kAny>());
}
template <class F>
cudaError_t with_lanes(int d, Pairs pairs, F f) {
    return d > 128 ? with_pairs<32>(pairs, f) : d > 64 ? with_pairs<16>(pairs, f) : with_pairs<8>(pairs, f);
}

}  // namespace

cudaError_t attn_heads_set_smem_limit() {
    cudaError_t e = cudaSuccess;
    for (const int d : {64, 128, 256})
        for (const Pairs pairs : {kHalves, kAdjacent, kAny})
            if (e == cudaSuccess)
                e = with_lanes(d, pairs, [](auto l, auto how) {
                    return cudaFuncSetAttribute(kv_append_kernel<l(), how()>,
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, kHeldBytes);
                });
    return e;
}

cudaError_t launch_norm_rope(const HeadRows &q, const HeadRows &k, const int *positions, const NormRope &how,
                             int tokens, int d, uint16_t *q_out, uint16_t *k_out, unsigned *err, int sms,
                             cudaStream_t stream) {
    return with_lanes(d, pairs_of(how, q.vec && k.vec), [&](auto l, auto pairs) {
        return norm_rope_l<l(), pairs()>(q, k, positions, how, tokens, d, q_out, k_out, err, sms, stream);
    });
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
    p.page_span = kv_page_span(n.max_q, c.page);
    return with_lanes(c.d, pairs_of(how, (q.heads == 0 || q.vec) && k.vec && v.vec),
                      [&](auto l, auto pairs) { return append_l<l(), pairs()>(p, stream); });
}

}  // namespace nvfp4
