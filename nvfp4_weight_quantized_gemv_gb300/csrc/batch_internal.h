// batch_internal.h -- declarations shared by the kernels that keep a batch of
// requests going (block tables, verification of drafts) and their entry
// points.  Not installed, not part of the C ABI.
#pragma once

#include "attn_internal.h"

namespace nvfp4 {

// kv_tables.cu
constexpr int kTablesMaxBatch = 8192;  // its sums lie in shared memory
struct TablesParams {
    int *table;
    long long table_stride;
    int width, batch, page_log2;
    int *pages;  // ring
    int ring;
    const long long *span;
    long long *span_out;
    const int *held, *kept, *kv, *q;  // kept may be nullptr
    int *held_out;
    int tokens;
    int *cu, *new_lens, *positions;
    long long *slots;
    unsigned *err;
};
cudaError_t tables_set_smem_limit();
cudaError_t launch_kv_tables(const TablesParams &p, cudaStream_t stream);

// verify.cu
struct VerifyParams {
    const float *target, *draft;  // draft may be nullptr
    long long target_stride, draft_stride;
    int vocab, batch, rows;
    const int *tokens, *cu, *kv;  // kv may be nullptr
    const float *u, *pick;
    int *out, *accepted, *next, *new_lens;
    unsigned *err;
};
cudaError_t launch_verify_drafts(const VerifyParams &p, cudaStream_t stream);

}  // namespace nvfp4
