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
// Attention behind shared prefixes: a group's rows over its prefix (the prompt
// kernel) and each sequence's over its own tokens (in chunks) leave parts, which
// a last kernel joins.  A small kernel ahead of them makes their records.
struct alignas(16) SharedSeq {
    int t0, q_len, kv_len;  // rows, and the tokens that they are multiplied with here
    int row, page0;         // where its pages begin in the block table
    int group;              // of a sequence: its group, -1 if it shares nothing
    int chunks, first_item; // of kv_len, and the number of the first one's item
    int parts;              // where its parts begin, in rows: [kv head][chunk][row]
    int units;              // of a group: its first unit in the prompt kernel's count, or its first CTA
    int split;              // of a group: CTAs of each of its blocks, 0 where they share units
    int pad;
};
struct alignas(16) SharedHead {
    int items, chunk;  // of all sequences' own tokens, and tokens of a chunk
    int next;          // items taken besides those that warps begin with
    int ctas;          // that share the prompt kernel's units
    int units;         // of all groups
    int pad[3];
};
struct alignas(16) SharedWalk {  // the prompt kernel's
    int b, h, rb, tile, t0, q_len, kv_len, tiles;
    int left, pad[3];
};
constexpr int kSharedMaxGroups = 2048;
struct SharedPlan {
    KvBatch n;
    const int *group_cu, *prefix_lens;
    int groups, max_group_tokens;
    int page_log2, heads, g, d;
    int rows_chunk;         // query rows that a chunk is multiplied with at a time
    float unit_steps;       // what a unit of the prompt kernel costs, in steps of 16 tokens of a chunk
    int chunk_warps;        // of an SM, that take chunks
    // A chunk's least tokens: of all blocks' tokens, so that there are few chunks in turns; of the prompt kernel's units; of
    // all rows' tokens, so that there is room for the parts.
    float of_steps, of_units, of_rows;
    int room;               // rows of all parts
    SharedHead *head;
    SharedSeq *prefixes, *own;  // [groups], [n.b]
    int *first;                 // [n.b + 1] first items
    SharedWalk *walks;          // [ctas]
    int ctas;
    unsigned *err;
};
// The prompt kernel's pass over the prefixes: the groups are its sequences, a
// row sees all tokens, and all results are parts: of blocks of several CTAs in
// `partials`, of others here.
struct SharedParams : AttnParams {
    const SharedSeq *seqs;
    const SharedWalk *walks;
    float *rows;  // [token][query head][head_dim + 4]
};
// attn_decode.cu
cudaError_t attn_decode_set_smem_limit(int smem_optin);
cudaError_t launch_attn_decode(const CUtensorMap &k, const CUtensorMap &v, const AttnParams &p, int smem_optin,
                               cudaStream_t stream);
// attn_prompt.cu
cudaError_t attn_prompt_set_smem_limit(int smem_optin);
cudaError_t launch_attn_prompt(const CUtensorMap &k, const CUtensorMap &v, const AttnParams &p, cudaStream_t stream);
cudaError_t launch_attn_prompt_pass(const CUtensorMap &k, const CUtensorMap &v, const SharedParams &p, cudaStream_t stream);
// attn_chunks.cu
struct ChunkParams : AttnParams {
    SharedHead *head;
    const SharedSeq *own;
    const int *first;
    float *parts;
    int room;  // rows of parts
};
cudaError_t attn_chunks_set_smem_limit();
inline int attn_chunk_rows(int rows) { return rows <= 8 ? 8 : 16; }
int attn_chunk_warps(int d, bool eight);  // of an SM
cudaError_t launch_attn_chunks(const ChunkParams &p, cudaStream_t stream);
// attn_shared.cu
struct SharedJoin : AttnParams {
    const SharedHead *head;
    const SharedSeq *prefixes, *own;
    const float *parts, *rows;
    int room;
};
cudaError_t attn_shared_set_smem_limit();
cudaError_t launch_attn_shared_plan(const SharedPlan &p, cudaStream_t stream);
cudaError_t launch_attn_shared_join(const SharedJoin &p, cudaStream_t stream);
// Whether a call with at most `rows` query rows a kv head takes the kernel for
// few rows: up to 16, its accumulators' and conversions' limit.  (16 sequences
// of 8192 tokens, 4 kv heads of 128: 8 rows 30 us there and 43 us in the kernel
// for prompts, 16 rows 38 and 43; heads of 256: 53 and 113, 58 and 111.  With 32
// rows a block it took 109 us for eight sequences of 25 rows over up to 16384
// tokens, the kernel for prompts takes 57.)
inline bool attn_few_rows(int rows) { return rows <= 16; }

}  // namespace nvfp4
