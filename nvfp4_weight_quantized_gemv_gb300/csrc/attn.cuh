// attn.cuh -- device building blocks shared by the attention kernels: tensor
// loads of the paged cache, conversions and the f16 tensor-core product.
#pragma once

#include "attn_internal.h"
#include "ptx.cuh"

#include <cuda_bf16.h>

namespace nvfp4 {

__device__ __forceinline__ float bf16_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float exp2_approx(float x) {  // 2 ulp
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / (1 + exp(-x)) to a few ulp (the result is rounded to bf16).
__device__ __forceinline__ float sigmoid(float x) {
    return __fdividef(1.f, 1.f + exp2_approx(-1.4426950408889634f * x));
}
// 2^e for an integer e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((127 + e) << 23); }

// d = a * b + c on pairs, sums and products of pairs.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
        " add.rn.f32x2 w, x, y;\n mov.b64 {%0, %1}, w;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
        " mul.rn.f32x2 w, x, y;\n mov.b64 {%0, %1}, w;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Four E4M3 codes -> two f16x2 (exact).
__device__ __forceinline__ void e4m3x4_f16(uint32_t v, uint32_t &lo, uint32_t &hi) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n"
        " cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}

// D[16x8] += A[16x16] B[16x8], f16 operands, fp32 accumulation.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The transpose of an 8x8 matrix of 16-bit entries held two a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}

// TMA box of the cache: entries x.. of slots y.., head z, page w.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void *tmap, int x, int y, int z, int w, uint32_t bar,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "l"(policy)
        : "memory");
}

// Orders what the kernel ahead wrote by plain stores before this thread's TMA loads.
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// Registers a thread of this warpgroup may use from here on (all four warps
// execute it; an increase waits until others have given theirs up).
template <int N>
__device__ __forceinline__ void set_max_regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_max_regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t pred;
    asm volatile(
        "{\n .reg .b32 r;\n .reg .pred p;\n elect.sync r|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(pred));
    return pred != 0;
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

constexpr int kWeightLift = 8;  // the products' weights are 2^8 at the running maximum

// The partial result of block [ub, ..) in CTA c of C, which share U units.
__device__ __forceinline__ float *attn_part(const AttnParams &p, int c, long long ub, long long U, long long C) {
    return p.partials + ((size_t)c * 2 + (c * U / C >= ub ? 0 : 1)) * p.slot_floats;
}

// What the weighted sums (in units of 2^(m - kWeightLift)) are multiplied by,
// for the weights' total `sum` (in units of 2^n), dm = m - n: 0 for a row that
// saw no token, NaN where the total is.  A scale of values of 2^100 and a
// reference n that lies 40 below the row's maximum (sum is 2^40 then) make dm
// 141, past the range of fp32, where the quotient is not: 64 of it go to the sum.
__device__ __forceinline__ float attn_inverse(float dm, float sum) {
    const float less = dm > 64.f ? 64.f : 0.f;
    return sum == 0.f ? 0.f : exp2_approx(dm - less - kWeightLift) / (sum * exp2_approx(-less));
}

// Entries d .. d + 3 of query row `row` of its sequence's rows (row = token *
// G + head): the weighted sums v times `inv`, gated, rounded.  A row that saw no
// token (inv == 0) is zero whatever its gate holds.
__device__ __forceinline__ void attn_store4(const AttnParams &p, int t0, int kvh, int row, int rows, int d, float4 v,
                                            float inv) {
    if (row >= rows || d >= p.c.d) return;
    const int i = row / p.g, h = kvh * p.g + row - i * p.g;
    float y[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
    if (p.gate.p && inv != 0.f) {
        const uint16_t *const gp = p.gate.p + (t0 + i) * p.gate.ts + h * p.gate.hs + d;
        uint16_t z[4];
        if (p.gate.vec) {
            const uint2 w = *reinterpret_cast<const uint2 *>(gp);
            z[0] = (uint16_t)w.x;
            z[1] = (uint16_t)(w.x >> 16);
            z[2] = (uint16_t)w.y;
            z[3] = (uint16_t)(w.y >> 16);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = gp[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] *= sigmoid(bf16_f32(z[e]));
    }
    *reinterpret_cast<uint2 *>(p.y + ((size_t)(t0 + i) * p.q.heads + h) * p.c.d + d) =
        make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
}

// Eight bf16 entries, by one load where alignment allows it.
__device__ __forceinline__ uint4 load_rows8(const uint16_t *p, int vec) {
    if (vec) return *reinterpret_cast<const uint4 *>(p);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = (uint32_t)p[2 * e] | ((uint32_t)p[2 * e + 1] << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight entries of a row: sums times `inv`, gated (not where inv == 0), rounded.
__device__ __forceinline__ void attn_store8(uint16_t *yp, bool gated, const uint4 &gate, const uint32_t *v, float inv) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(v[e]) * inv;
    if (gated && inv != 0.f) {
        const uint32_t z[4] = {gate.x, gate.y, gate.z, gate.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[2 * e] *= sigmoid(__uint_as_float(z[e] << 16));
            y[2 * e + 1] *= sigmoid(__uint_as_float(z[e] & 0xFFFF0000u));
        }
    }
    *reinterpret_cast<uint4 *>(yp) =
        make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
}

}  // namespace nvfp4
