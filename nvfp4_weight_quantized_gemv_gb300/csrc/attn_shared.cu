// attn_shared.cu -- attention for a batch whose sequences share long prefixes:
// the sequences of its two passes.
//
// With (n, l, y) a row's reference, weights' total in units of 2^n and mean of
// values over the prefix, and (m, s, z) the same over its sequence's own tokens,
//
//     result = (l 2^(n - t) y + s 2^(m - t) z) / (l 2^(n - t) + s 2^(m - t)),   t = max(n, m).
//
// The first pass takes a group's rows, neighbours in the batch, as those of one
// sequence that see all of the prefix: 64 sequences of four query heads a kv head
// are two blocks of 128 rows for the tensor core, where 64 passes over the prefix
// would each be bound by its bytes.  The second pass is attention as it is
// without prefixes, over tables and lengths that begin behind them; its last
// step, wherever a row is finished, takes the first pass's result in.
//
// What is shared of a prefix is what every token of the group sees, whole pages
// and whole tiles of 128 tokens of it: so the first pass needs no masks, and what
// is left of a prefix is read with each sequence's own tokens.
#include "attn_internal.h"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kWhole = 128;  // tokens of a tile

// A CTA a group, and one for the sequences of no group.
__global__ void __launch_bounds__(kThreads) attn_shared_plan_kernel(const SharedPlan s, const KvBatch n, const int page_log2,
                                                                    unsigned *err) {
    __shared__ int sh_start, sh_first, sh_active;
    const int group = blockIdx.x;
    griddep_wait();
    bool ok = true;
    for (int g = threadIdx.x; g < s.groups; g += kThreads) {
        const int c0 = s.group_cu[g], c1 = s.group_cu[g + 1];
        ok = ok && c0 >= 0 && c1 >= c0 && c1 <= n.b;
    }
    if (threadIdx.x == 0) {
        sh_start = sh_first = 0x7FFFFFFF;
        sh_active = 0;
    }
    ok = __syncthreads_and(ok);
    if (!ok && group == 0 && threadIdx.x == 0) atomicOr(err, kDevErrAttnInput);
    auto own = [&](int b, int shared) {  // the record of sequence b behind `shared` tokens
        int t0, q_len, kv_len;
        if (!kv_sequence(n, b, &t0, &q_len, &kv_len)) atomicOr(err, kDevErrAttnInput);
        if (kv_len == 0) shared = 0;
        s.own[b] = SharedSeq{t0, q_len, kv_len - shared, b, shared >> page_log2, {0, 0, 0}};
    };
    if (!ok || group == s.groups) {
        const int first = ok ? s.group_cu[0] : n.b, behind = ok ? s.group_cu[s.groups] : n.b;
        if (!ok && group < s.groups && threadIdx.x == 0) s.prefixes[group] = SharedSeq{0, 0, 0, 0, 0, {0, 0, 0}};
        if (group == s.groups) {
            for (int b = threadIdx.x; b < first; b += kThreads) own(b, 0);
            for (int b = behind + threadIdx.x; b < n.b; b += kThreads) own(b, 0);
        }
        return;
    }
    const int b0 = s.group_cu[group], b1 = s.group_cu[group + 1];
    int length = s.prefix_lens[group];
    if (length < 0 || length > n.max_kv) {
        if (threadIdx.x == 0) atomicOr(err, kDevErrAttnInput);
        length = 0;
    }
    bool rows_ok = true;  // the group's rows are neighbours
    for (int b = b0 + threadIdx.x; b < b1; b += kThreads) {
        const int c0 = n.cu[b], c1 = n.cu[b + 1];
        rows_ok = rows_ok && c0 >= 0 && c1 >= c0 && c1 <= n.tokens && c1 - c0 <= n.max_q;
        int t0, q_len, kv_len;
        kv_sequence(n, b, &t0, &q_len, &kv_len);
        if (q_len > 0 && kv_len > 0) {  // others see nothing of the prefix
            atomicMin(&sh_start, max(0, kv_len - q_len));
            atomicMin(&sh_first, b);
            atomicAdd(&sh_active, 1);
        }
    }
    rows_ok = __syncthreads_and(rows_ok);
    const int t0 = b1 > b0 ? n.cu[b0] : 0, tokens = b1 > b0 && rows_ok ? n.cu[b1] - t0 : 0;
    const int unit = max(kWhole, 1 << page_log2);
    const int shared = rows_ok && sh_active > 1 && tokens <= s.max_group_tokens ? min(length, sh_start) / unit * unit : 0;
    if (threadIdx.x == 0)
        s.prefixes[group] = shared > 0 ? SharedSeq{t0, tokens, shared, sh_first, 0, {0, 0, 0}} : SharedSeq{0, 0, 0, 0, 0, {0, 0, 0}};
    for (int b = b0 + threadIdx.x; b < b1; b += kThreads) own(b, shared);
}

}  // namespace

cudaError_t launch_attn_shared_plan(const SharedPlan &s, const KvBatch &n, int page_log2, unsigned *err, cudaStream_t stream) {
    return launch_behind(attn_shared_plan_kernel, dim3((unsigned)s.groups + 1), kThreads, 0, stream, s, n, page_log2, err);
}

}  // namespace nvfp4
