// abi_batch.cu -- C entry points of the block tables and of the verification of
// drafted tokens: argument checks and launch.
#include "abi_internal.h"
#include "batch_internal.h"

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_kv_tables(const nvfp4_kv_pages *pages, int batch, const int32_t *kv_lens,
                                        const int32_t *q_lens, int tokens, int32_t *cu_q, int32_t *new_lens,
                                        int32_t *positions, int64_t *slots, cudaStream_t stream) {
    if (!pages) return fail(NVFP4_ERR_INVALID_ARG, "null nvfp4_kv_pages");
    if (batch < 0 || batch > kTablesMaxBatch || tokens < 0 || tokens > (1 << 30))
        return fail(NVFP4_ERR_INVALID_ARG, "batch = %d (0..%d), tokens = %d (0..2^30) out of range", batch,
                    kTablesMaxBatch, tokens);
    int log2 = 4;
    while (log2 < 8 && (1 << log2) != pages->page_size) ++log2;
    if ((1 << log2) != pages->page_size)
        return fail(NVFP4_ERR_INVALID_ARG, "page_size = %d must be 16, 32, 64, 128 or 256", pages->page_size);
    if (pages->table_width < 1 || pages->table_width > (1 << 26) || pages->table_stride < 0 || pages->ring < 1 ||
        pages->ring > (1 << 30) || (batch > 1 && pages->table_stride < pages->table_width))
        return fail(NVFP4_ERR_INVALID_ARG, "pages: table_width = %d, table_stride = %lld, ring = %d out of range",
                    pages->table_width, pages->table_stride, pages->ring);
    if (!pages->free_pages || !pages->span || !pages->span_out || !cu_q || (tokens > 0 && (!positions || !slots)) ||
        (batch > 0 && (!pages->block_table || !pages->held || !pages->held_out || !kv_lens || !q_lens || !new_lens)))
        return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
    for (const void *p : {(const void *)pages->block_table, (const void *)pages->free_pages, (const void *)pages->held,
                          (const void *)pages->held_out, (const void *)pages->kept, (const void *)kv_lens,
                          (const void *)q_lens, (const void *)cu_q, (const void *)new_lens, (const void *)positions})
        if (!aligned(p, 4)) return fail(NVFP4_ERR_MISALIGNED, "32-bit arrays must be 4-byte aligned");
    for (const void *p : {(const void *)pages->span, (const void *)pages->span_out, (const void *)slots})
        if (!aligned(p, 8)) return fail(NVFP4_ERR_MISALIGNED, "span and slots must be 8-byte aligned");
    int dev = 0;
    DeviceState *d = nullptr;
    nvfp4_status st = current_device(&dev, &d);
    if (st != NVFP4_OK) return st;
    TablesParams p;
    p.table = pages->block_table;
    p.table_stride = pages->table_stride;
    p.width = pages->table_width;
    p.batch = batch;
    p.page_log2 = log2;
    p.pages = pages->free_pages;
    p.ring = pages->ring;
    p.span = reinterpret_cast<const long long *>(pages->span);
    p.span_out = reinterpret_cast<long long *>(pages->span_out);
    p.held = pages->held;
    p.kept = pages->kept;
    p.kv = kv_lens;
    p.q = q_lens;
    p.held_out = pages->held_out;
    p.tokens = tokens;
    p.cu = cu_q;
    p.new_lens = new_lens;
    p.positions = positions;
    p.slots = reinterpret_cast<long long *>(slots);
    p.err = d->err_word;
    cudaError_t e = launch_kv_tables(p, stream);
    return e == cudaSuccess ? NVFP4_OK : cuda_fail(e, "block tables launch");
}

extern "C" nvfp4_status nvfp4_verify_drafts(const nvfp4_draft_rows *rows, const int32_t *cu_q, const int32_t *kv_lens,
                                            const float *u_accept, const float *u_next, int batch, int32_t *out_tokens,
                                            int32_t *accepted, int32_t *next, int32_t *new_lens, cudaStream_t stream) {
    if (!rows) return fail(NVFP4_ERR_INVALID_ARG, "null nvfp4_draft_rows");
    if (batch < 0 || batch > 65535 || rows->tokens < 0 || rows->tokens > (1 << 30))
        return fail(NVFP4_ERR_INVALID_ARG, "batch = %d (0..65535), tokens = %d (0..2^30) out of range", batch, rows->tokens);
    if (rows->vocab < 1 || rows->vocab > (1 << 30))
        return fail(NVFP4_ERR_INVALID_ARG, "vocab = %d must be in [1, 2^30]", rows->vocab);
    if (rows->target_stride < 0 || rows->draft_stride < 0) return fail(NVFP4_ERR_INVALID_ARG, "negative stride");
    if (batch == 0) return NVFP4_OK;
    if (!cu_q || !accepted || !next || (kv_lens && !new_lens) || !u_next ||
        (rows->tokens > 0 && (!rows->target || !rows->ids || !u_accept || !out_tokens)))
        return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
    for (const void *p : {(const void *)rows->target, (const void *)rows->draft, (const void *)rows->ids, (const void *)cu_q,
                          (const void *)kv_lens, (const void *)u_accept, (const void *)u_next, (const void *)out_tokens,
                          (const void *)accepted, (const void *)next, (const void *)new_lens})
        if (!aligned(p, 4)) return fail(NVFP4_ERR_MISALIGNED, "arrays must be 4-byte aligned");
    int dev = 0;
    DeviceState *d = nullptr;
    nvfp4_status st = current_device(&dev, &d);
    if (st != NVFP4_OK) return st;
    VerifyParams p;
    p.target = rows->target;
    p.draft = rows->draft;
    p.target_stride = rows->target_stride;
    p.draft_stride = rows->draft_stride;
    p.vocab = rows->vocab;
    p.batch = batch;
    p.rows = rows->tokens;
    p.tokens = rows->ids;
    p.cu = cu_q;
    p.kv = kv_lens;
    p.u = u_accept;
    p.pick = u_next;
    p.out = out_tokens;
    p.accepted = accepted;
    p.next = next;
    p.new_lens = new_lens;
    p.err = d->err_word;
    cudaError_t e = launch_verify_drafts(p, stream);
    return e == cudaSuccess ? NVFP4_OK : cuda_fail(e, "verification launch");
}
