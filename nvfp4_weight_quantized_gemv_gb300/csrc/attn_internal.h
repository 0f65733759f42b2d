// attn_internal.h -- declarations shared by the attention operators' kernels
// (norm and rotation, the paged 8-bit cache, attention over it) and their
// entry points.  Not installed, not part of the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace nvfp4 {

constexpr unsigned kDevErrAttnInput = 256u;  // device error word: a position, length or page number out of range
constexpr int kAttnMaxHeadDim = 256;

// bf16 rows [tokens][heads][head_dim] with strides in elements.
struct HeadRows {
    const uint16_t *p;
    long long ts, hs;
    int heads;
    int vec;  // 1: base and strides allow 16-byte loads
};

struct NormRope {
    const uint16_t *qw, *kw;
    const float *cs;
    float eps;
    int positions, rot, interleaved;
    int cs_vec;  // 1: 16-byte loads of the table (rot a multiple of 8, 16-byte aligned)
    int qw_vec, kw_vec;  // 1: 16-byte loads of the weights
};

struct KvCache {
    uint8_t *k, *v;
    float *ks, *vs;
    long long ps, hs, ts;  // byte strides of page, head, slot
    int pages, heads, page, page_log2, d;
};

struct KvBatch {
    const int *table, *cu, *kv;
    int b, table_stride, tokens, max_q, max_kv;
};

#ifdef __CUDACC__
// Lengths of sequence b: its first token of the call, how many it brings, how
// many it holds.  One whose cu_q cannot be used brings nothing, one whose
// kv_lens cannot be used holds nothing; false in both cases.
__device__ __forceinline__ bool kv_sequence(const KvBatch &n, int b, int *t0, int *q_len, int *kv_len) {
    const int c0 = n.cu[b], c1 = n.cu[b + 1], kv = n.kv[b];
    const bool cu_ok = c0 >= 0 && c1 >= c0 && c1 <= n.tokens && c1 - c0 <= n.max_q;
    const bool kv_ok = kv >= 0 && kv <= n.max_kv;
    *t0 = cu_ok ? c0 : 0;
    *q_len = cu_ok ? c1 - c0 : 0;
    *kv_len = kv_ok ? kv : 0;
    return cu_ok && kv_ok;
}
#endif

// Launches a kernel that may be set up, and its CTAs placed, while the one ahead
// in the stream ends: it waits for that one (griddep_wait) before it touches
// memory.  About 1 us a call in a chain of short ones.
template <class... P, class... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                          const A &...args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// attn_heads.cu
// Pages that `tokens` consecutive tokens can touch (tokens + page may pass 2^31).
inline int kv_page_span(int tokens, int page) { return (int)(((long long)tokens + page - 2) / page + 1); }
cudaError_t attn_heads_set_smem_limit();
cudaError_t launch_norm_rope(const HeadRows &q, const HeadRows &k, const int *positions, const NormRope &how,
                             int tokens, int d, uint16_t *q_out, uint16_t *k_out, unsigned *err, int sms,
                             cudaStream_t stream);
cudaError_t launch_kv_append(const HeadRows &q, const HeadRows &k, const HeadRows &v, const NormRope &how,
                             const KvCache &c, const KvBatch &n, uint16_t *q_out, unsigned *err, cudaStream_t stream);

// Attention over the paged cache.
struct AttnParams {
    HeadRows q, gate;  // gate.p == nullptr: none
    KvCache c;
    KvBatch n;
    uint16_t *y;
    float scale_log2;  // softmax scale times log2(e)
    int g;             // query heads per kv head
    unsigned g_magic;  // ceil(2^32 / g), 0 for g == 1
#ifdef __CUDACC__
    // x / g for x * g < 2^32.
    __device__ __forceinline__ int g_div(int x) const { return g_magic ? (int)__umulhi((unsigned)x, g_magic) : x; }
#endif
    unsigned *err;
    float *partials;     // [ctas][2][slot_floats]: a CTA's first and last block, where other CTAs have parts of it
    int slot_floats;
    int ctas;            // persistent grid
};
// Workspace: the partial results, then a record a CTA about the block that it
// begins and others continue.  A slot holds the (maxima of w and s, sum) of a
// block's rows and their weighted sums.
constexpr int kAttnSlotFloats = 128 * (256 + 4);
constexpr int kAttnJoinBytes = 64;
inline size_t attn_workspace_bytes(int sms) {
    return (size_t)sms * (2 * kAttnSlotFloats * sizeof(float) + kAttnJoinBytes);
}
// attn_decode.cu
cudaError_t attn_decode_set_smem_limit(int smem_optin);
cudaError_t launch_attn_decode(const CUtensorMap &k, const CUtensorMap &v, const AttnParams &p, int smem_optin,
                               cudaStream_t stream);
// attn_prompt.cu
cudaError_t attn_prompt_set_smem_limit(int smem_optin);
cudaError_t launch_attn_prompt(const CUtensorMap &k, const CUtensorMap &v, const AttnParams &p, cudaStream_t stream);
// Whether a call with at most `rows` query rows a kv head takes the kernel for
// few rows: up to 16, its accumulators' and conversions' limit.  (16 sequences
// of 8192 tokens, 4 kv heads of 128: 8 rows 30 us there and 43 us in the kernel
// for prompts, 16 rows 38 and 43; heads of 256: 53 and 113, 58 and 111.  With 32
// rows a block it took 109 us for eight sequences of 25 rows over up to 16384
// tokens, the kernel for prompts takes 57.)
inline bool attn_few_rows(int rows) { return rows <= 16; }

}  // namespace nvfp4
