// attn_paged.cu -- causal attention over the paged 8-bit cache.
//
// One warp for every (token, query head): the query in registers (eight
// entries a lane), one pass over the visible tokens with the running maximum
// m and sum l of the softmax,
//
//     s = scale * q . K[j],  m' = max(m, s),  l = l 2^(m - m') + 2^(s - m'),
//     o = o 2^(m - m') + 2^(s - m') V[j].
#include "attn_internal.h"
#include "ptx.cuh"

#include <cuda_bf16.h>

namespace nvfp4 {

namespace {

constexpr int kSimpleWarps = 8;

__device__ __forceinline__ float bf16_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

__device__ __forceinline__ void code8(const uint8_t *p, float (&x)[8]) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    const uint32_t w[4] = {v.x, v.x >> 16, v.y, v.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t h = e4m3x2_to_f16x2(w[i]);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__global__ void __launch_bounds__(kSimpleWarps * 32) attn_simple_kernel(const AttnParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * 8;
    const int b = blockIdx.y;
    const int hq = p.q.heads;
    const long long item = (long long)blockIdx.x * kSimpleWarps + warp;
    const int i = (int)(item / hq), h = (int)(item % hq);
    int t0, q_len, kv_len;
    if (!kv_sequence(p.n, b, &t0, &q_len, &kv_len) && lane == 0) atomicOr(p.err, kDevErrAttnInput);
    if (i >= q_len) return;
    const int D = p.c.d, kvh = h / p.g, seen = kv_len - q_len + i + 1;
    const bool on = e0 < D;
    const uint16_t *qp = p.q.p + (t0 + i) * p.q.ts + h * p.q.hs + e0;
    float q[8], o[8], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        q[k] = on ? bf16_f32(qp[k]) * p.scale_log2 : 0.f;
        o[k] = 0.f;
    }
    const int *table = p.n.table + (size_t)b * p.n.table_stride;
    for (int j = 0; j < seen; ++j) {
        const int page = table[j >> p.c.page_log2];
        const bool there = page >= 0 && page < p.c.pages;
        if (!there && lane == 0) atomicOr(p.err, kDevErrAttnInput);
        const size_t at = (size_t)(there ? page : 0) * p.c.ps + (size_t)kvh * p.c.hs +
                          (size_t)(j & (p.c.page - 1)) * p.c.ts + e0;
        const size_t sc = (size_t)(there ? page : 0) * p.c.heads + kvh;
        float k[8], v[8], s = 0.f;
#pragma unroll
        for (int x = 0; x < 8; ++x) k[x] = v[x] = 0.f;
        if (on && there) {
            code8(p.c.k + at, k);
            code8(p.c.v + at, v);
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) s = fmaf(q[x], k[x], s);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= p.c.ks[sc];
        const float top = fmaxf(m, s), f = exp2f(m - top), w = exp2f(s - top), wv = w * p.c.vs[sc];
        l = fmaf(l, f, w);
#pragma unroll
        for (int x = 0; x < 8; ++x) o[x] = fmaf(o[x], f, wv * v[x]);
        m = top;
    }
    if (!on) return;
    const size_t row = ((size_t)(t0 + i) * hq + h) * D + e0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float v = seen > 0 ? o[k] / l : 0.f;
        if (p.gate.p) v = v / (1.f + expf(-bf16_f32(p.gate.p[(t0 + i) * p.gate.ts + h * p.gate.hs + e0 + k])));
        const __nv_bfloat16 r = __float2bfloat16_rn(v);
        p.y[row + k] = *reinterpret_cast<const uint16_t *>(&r);
    }
}

}  // namespace

cudaError_t attn_set_smem_limit(int) { return cudaSuccess; }

size_t attn_workspace_bytes(int) { return 256; }

cudaError_t launch_attn(const AttnParams &p, cudaStream_t stream) {
    const long long items = (long long)p.n.max_q * p.q.heads;
    const dim3 grid((unsigned)((items + kSimpleWarps - 1) / kSimpleWarps), (unsigned)p.n.b);
    attn_simple_kernel<<<grid, kSimpleWarps * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace nvfp4
