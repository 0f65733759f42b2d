// abi_attn.cu -- C entry points of the attention operators: argument checks,
// workspace and launch.
#include "abi_internal.h"
#include "attn_internal.h"
#include "attn_units.h"

#include <cmath>

namespace nvfp4 {

static nvfp4_status check_head_dim(int d) {
    if (d < 16 || d > kAttnMaxHeadDim || d % 16 != 0)
        return fail(NVFP4_ERR_INVALID_ARG, "head_dim = %d must be a multiple of 16 in [16, %d]", d, kAttnMaxHeadDim);
    return NVFP4_OK;
}

static nvfp4_status take_rows(const nvfp4_head_rows *r, const char *name, HeadRows *out) {
    *out = HeadRows{nullptr, 0, 0, 0, 0};
    if (!r) return NVFP4_OK;
    if (!r->p) return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", name);
    if (r->heads < 1 || r->heads > 65536)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: heads = %d out of range", name, r->heads);
    if (r->token_stride < 0 || r->head_stride < 0)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: negative stride", name);
    if (!aligned(r->p, 2)) return fail(NVFP4_ERR_MISALIGNED, "%s must be 2-byte aligned", name);
    out->p = r->p;
    out->ts = r->token_stride;
    out->hs = r->head_stride;
    out->heads = r->heads;
    out->vec = aligned(r->p, 16) && r->token_stride % 8 == 0 && r->head_stride % 8 == 0;
    return NVFP4_OK;
}

static nvfp4_status take_norm_rope(const nvfp4_norm_rope *how, int d, NormRope *out) {
    if (!how) return fail(NVFP4_ERR_INVALID_ARG, "null nvfp4_norm_rope");
    if (how->rot < 0 || how->rot > d || how->rot % 2 != 0)
        return fail(NVFP4_ERR_INVALID_ARG, "rot = %d must be even and in [0, head_dim = %d]", how->rot, d);
    if (how->rot > 0 && (!how->cos_sin || how->table_positions < 1))
        return fail(NVFP4_ERR_INVALID_ARG, "rot = %d needs a table of positions", how->rot);
    if (how->interleaved != 0 && how->interleaved != 1)
        return fail(NVFP4_ERR_INVALID_ARG, "interleaved must be 0 or 1");
    if ((how->q_weight || how->k_weight) && !(how->eps >= 0.f && std::isfinite(how->eps)))
        return fail(NVFP4_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (!aligned(how->cos_sin, 4) || !aligned(how->q_weight, 2) || !aligned(how->k_weight, 2))
        return fail(NVFP4_ERR_MISALIGNED, "the table must be 4-byte aligned, the weights 2-byte");
    out->qw = how->q_weight;
    out->kw = how->k_weight;
    out->cs = how->cos_sin;
    out->eps = how->eps;
    out->positions = how->table_positions;
    out->rot = how->rot;
    out->interleaved = how->interleaved;
    out->cs_vec = how->rot % 8 == 0 && aligned(how->cos_sin, 16);
    out->qw_vec = aligned(how->q_weight, 16);
    out->kw_vec = aligned(how->k_weight, 16);
    return NVFP4_OK;
}

static nvfp4_status take_cache(const nvfp4_kv_cache *c, KvCache *out) {
    if (!c) return fail(NVFP4_ERR_INVALID_ARG, "null nvfp4_kv_cache");
    nvfp4_status st = check_head_dim(c->head_dim);
    if (st != NVFP4_OK) return st;
    if (!c->k || !c->v || !c->k_scale || !c->v_scale) return fail(NVFP4_ERR_INVALID_ARG, "cache: null pointer");
    if (c->pages < 1 || c->kv_heads < 1 || c->kv_heads > 65536)
        return fail(NVFP4_ERR_INVALID_ARG, "cache: pages = %d, kv_heads = %d out of range", c->pages, c->kv_heads);
    int log2 = 4;
    while (log2 < 8 && (1 << log2) != c->page_size) ++log2;
    if ((1 << log2) != c->page_size)
        return fail(NVFP4_ERR_INVALID_ARG, "page_size = %d must be 16, 32, 64, 128 or 256", c->page_size);
    // 2^39: a tensor map's strides are below 2^40 bytes
    const long long most = 1ll << 39;
    if (c->page_stride < 0 || c->head_stride < 0 || c->token_stride < c->head_dim || c->page_stride > most ||
        c->head_stride > most || c->token_stride > most)
        return fail(NVFP4_ERR_INVALID_ARG, "cache: strides %lld, %lld, %lld out of range", c->page_stride,
                    c->head_stride, c->token_stride);
    if (c->page_stride % 16 != 0 || c->head_stride % 16 != 0 || c->token_stride % 16 != 0 || !aligned(c->k, 16) ||
        !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return fail(NVFP4_ERR_MISALIGNED, "cache: codes and strides must be multiples of 16 bytes");
    *out = KvCache{c->k, c->v, c->k_scale, c->v_scale, c->page_stride, c->head_stride, c->token_stride,
                   c->pages, c->kv_heads, c->page_size, log2, c->head_dim};
    return NVFP4_OK;
}

// A view of the cache's codes for TMA: boxes of 128 entries (a swizzled row
// of a tile; entries past head_dim read as zeros) by up to 64 slots of a page.
// Through a small per-thread cache, as encoding a map is host work on every
// call's path; keyed by everything the map depends on.
static nvfp4_status cache_map(CUtensorMap *map, const uint8_t *codes, const KvCache &c) {
    struct Entry {
        const uint8_t *p;
        KvCache c;
        CUtensorMap map;
    };
    constexpr int kEntries = 64;
    static thread_local Entry cache[kEntries];
    static thread_local int used = 0, next = 0;
    for (int i = 0; i < used; ++i) {
        const Entry &e = cache[i];
        if (e.p == codes && e.c.ps == c.ps && e.c.hs == c.hs && e.c.ts == c.ts && e.c.pages == c.pages &&
            e.c.heads == c.heads && e.c.page == c.page && e.c.d == c.d) {
            *map = e.map;
            return NVFP4_OK;
        }
    }
    EncodeTiledFn fn;
    nvfp4_status st = get_encode_fn(&fn);
    if (st != NVFP4_OK) return st;
    const cuuint64_t dims[4] = {(cuuint64_t)c.d, (cuuint64_t)c.page, (cuuint64_t)c.heads, (cuuint64_t)c.pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.ts, (cuuint64_t)c.hs, (cuuint64_t)c.ps};
    const cuuint32_t box[4] = {128, (cuuint32_t)(c.page < 64 ? c.page : 64), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t *>(codes), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(NVFP4_ERR_CUDA, "cuTensorMapEncodeTiled (cache) failed (CUresult %d)", (int)r);
    Entry &e = cache[next];
    e = Entry{codes, c, *map};
    next = (next + 1) % kEntries;
    if (used < kEntries) ++used;
    return NVFP4_OK;
}

// NVFP4_OK and out->b == 0: nothing to do.
static nvfp4_status take_batch(const nvfp4_kv_batch *n, const KvCache &c, KvBatch *out) {
    if (!n) return fail(NVFP4_ERR_INVALID_ARG, "null nvfp4_kv_batch");
    if (n->batch < 0 || n->tokens < 0 || n->batch > 65535)
        return fail(NVFP4_ERR_INVALID_ARG, "batch = %d (0..65535), tokens = %d out of range", n->batch, n->tokens);
    *out = KvBatch{n->block_table, n->cu_q, n->kv_lens, n->batch, n->table_stride, n->tokens, n->max_q_len,
                   n->max_kv_len};
    if (n->batch == 0 || n->tokens == 0) {
        out->b = 0;
        return NVFP4_OK;
    }
    if (!n->block_table || !n->cu_q || !n->kv_lens) return fail(NVFP4_ERR_INVALID_ARG, "batch: null pointer");
    if (n->table_stride < 1 || n->max_q_len < 1 || n->max_kv_len < 0 || n->max_kv_len > (1 << 30) ||
        (long long)n->table_stride * c.page < n->max_kv_len)
        return fail(NVFP4_ERR_INVALID_ARG,
                    "batch: max_q_len = %d, max_kv_len = %d, table of %d pages of %d tokens out of range",
                    n->max_q_len, n->max_kv_len, n->table_stride, c.page);
    if (out->max_q > n->tokens) out->max_q = n->tokens;
    return NVFP4_OK;
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_qk_norm_rope(const nvfp4_head_rows *q, const nvfp4_head_rows *k,
                                           const int32_t *positions, const nvfp4_norm_rope *how, int tokens,
                                           int head_dim, uint16_t *q_out, uint16_t *k_out, cudaStream_t stream) {
    HeadRows qr, kr;
    NormRope nr;
    nvfp4_status st = check_head_dim(head_dim);
    if (st != NVFP4_OK) return st;
    if (tokens < 0) return fail(NVFP4_ERR_INVALID_ARG, "tokens = %d must be >= 0", tokens);
    if (!q) return fail(NVFP4_ERR_INVALID_ARG, "q: null pointer");
    if ((st = take_norm_rope(how, head_dim, &nr)) != NVFP4_OK) return st;
    if (tokens == 0) return NVFP4_OK;
    if ((st = take_rows(q, "q", &qr)) != NVFP4_OK || (st = take_rows(k, "k", &kr)) != NVFP4_OK) return st;
    if (!q_out || (k && !k_out) || (nr.rot > 0 && !positions))
        return fail(NVFP4_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned(q_out, 16) || (k && !aligned(k_out, 16)))
        return fail(NVFP4_ERR_MISALIGNED, "outputs must be 16-byte aligned");
    if ((long long)tokens * (qr.heads + kr.heads) > (1ll << 32))
        return fail(NVFP4_ERR_INVALID_ARG, "tokens * heads too large");
    int dev = 0;
    DeviceState *d = nullptr;
    if ((st = current_device(&dev, &d)) != NVFP4_OK) return st;
    cudaError_t e = launch_norm_rope(qr, kr, positions, nr, tokens, head_dim, q_out, k_out, d->err_word, d->sms, stream);
    return e == cudaSuccess ? NVFP4_OK : cuda_fail(e, "norm and rotation launch");
}

extern "C" nvfp4_status nvfp4_kv_append(const nvfp4_head_rows *q, const nvfp4_head_rows *k, const nvfp4_head_rows *v,
                                        const nvfp4_norm_rope *how, const nvfp4_kv_cache *cache,
                                        const nvfp4_kv_batch *batch, uint16_t *q_out, cudaStream_t stream) {
    HeadRows qr, kr, vr;
    NormRope nr;
    KvCache c;
    KvBatch n;
    nvfp4_status st;
    if ((st = take_cache(cache, &c)) != NVFP4_OK || (st = take_batch(batch, c, &n)) != NVFP4_OK ||
        (st = take_norm_rope(how, c.d, &nr)) != NVFP4_OK || n.b == 0)
        return st;
    if (!k || !v) return fail(NVFP4_ERR_INVALID_ARG, "k or v: null pointer");
    if ((st = take_rows(q, "q", &qr)) != NVFP4_OK || (st = take_rows(k, "k", &kr)) != NVFP4_OK ||
        (st = take_rows(v, "v", &vr)) != NVFP4_OK)
        return st;
    if (kr.heads != c.heads || vr.heads != c.heads)
        return fail(NVFP4_ERR_INVALID_ARG, "k has %d heads and v %d, the cache %d", kr.heads, vr.heads, c.heads);
    if (q && !q_out) return fail(NVFP4_ERR_INVALID_ARG, "q_out: null pointer");
    if (q && !aligned(q_out, 16)) return fail(NVFP4_ERR_MISALIGNED, "q_out must be 16-byte aligned");
    if (nr.rot > 0 && nr.positions < n.max_kv)
        return fail(NVFP4_ERR_INVALID_ARG, "a table of %d positions for max_kv_len = %d", nr.positions, n.max_kv);
    if ((long long)n.b * kv_page_span(n.max_q, c.page) * (2 * c.heads + qr.heads) > 0x7FFFFFFF)
        return fail(NVFP4_ERR_INVALID_ARG, "batch * pages * heads too large");
    int dev = 0;
    DeviceState *d = nullptr;
    if ((st = current_device(&dev, &d)) != NVFP4_OK) return st;
    cudaError_t e = launch_kv_append(qr, kr, vr, nr, c, n, q_out, d->err_word, stream);
    return e == cudaSuccess ? NVFP4_OK : cuda_fail(e, "append launch");
}

// Arguments that both attention entry points take; NVFP4_OK and p->n.b == 0: nothing to do.
static nvfp4_status take_attn(const nvfp4_head_rows *q, const nvfp4_kv_cache *cache, const nvfp4_kv_batch *batch, float scale,
                              const nvfp4_head_rows *gate, uint16_t *y, const void *workspace, AttnParams *p) {
    nvfp4_status st;
    if ((st = take_cache(cache, &p->c)) != NVFP4_OK || (st = take_batch(batch, p->c, &p->n)) != NVFP4_OK) return st;
    if (!(scale > 0.f) || !std::isfinite(scale))
        return fail(NVFP4_ERR_INVALID_ARG, "scale must be positive and finite");
    if (workspace && !aligned(workspace, 256))
        return fail(NVFP4_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (p->n.b == 0) return NVFP4_OK;
    if (!q || !y) return fail(NVFP4_ERR_INVALID_ARG, "q or y: null pointer");
    if ((st = take_rows(q, "q", &p->q)) != NVFP4_OK || (st = take_rows(gate, "gate", &p->gate)) != NVFP4_OK) return st;
    if (p->q.heads % p->c.heads != 0)
        return fail(NVFP4_ERR_INVALID_ARG, "%d query heads are no multiple of %d kv heads", p->q.heads, p->c.heads);
    if (gate && p->gate.heads != p->q.heads)
        return fail(NVFP4_ERR_INVALID_ARG, "gate has %d heads, q %d", p->gate.heads, p->q.heads);
    if (!aligned(y, 16)) return fail(NVFP4_ERR_MISALIGNED, "y must be 16-byte aligned");
    if ((long long)p->n.max_q * p->q.heads > (1 << 30))
        return fail(NVFP4_ERR_INVALID_ARG, "max_q_len * heads too large");
    p->y = y;
    p->scale_log2 = scale * 1.4426950408889634f;
    p->g = p->q.heads / p->c.heads;
    p->g_magic = p->g > 1 ? (unsigned)(((1ull << 32) + p->g - 1) / p->g) : 0;
    return NVFP4_OK;
}

static cudaError_t launch_attn(const CUtensorMap &k, const CUtensorMap &v, const AttnParams &p, int smem_optin,
                               cudaStream_t stream) {
    return attn_few_rows(p.n.max_q * p.g) ? launch_attn_decode(k, v, p, smem_optin, stream) : launch_attn_prompt(k, v, p, stream);
}

extern "C" nvfp4_status nvfp4_attn_paged(const nvfp4_head_rows *q, const nvfp4_kv_cache *cache,
                                         const nvfp4_kv_batch *batch, float scale, const nvfp4_head_rows *gate,
                                         uint16_t *y, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    AttnParams p;
    nvfp4_status st = take_attn(q, cache, batch, scale, gate, y, workspace, &p);
    if (st != NVFP4_OK || p.n.b == 0) return st;
    int dev = 0;
    DeviceState *d = nullptr;
    if ((st = current_device(&dev, &d)) != NVFP4_OK) return st;
    const size_t need = attn_workspace_bytes(d->sms);
    if (workspace) {
        if (workspace_bytes < need)
            return fail(NVFP4_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed", workspace_bytes, need);
    } else if ((st = stream_workspace(dev, stream, kWsAttn, need, &workspace)) != NVFP4_OK) {
        return st;
    }
    p.err = d->err_word;
    p.ctas = d->sms;
    p.partials = static_cast<float *>(workspace);
    p.slot_floats = kAttnSlotFloats;
    CUtensorMap map_k, map_v;
    if ((st = cache_map(&map_k, p.c.k, p.c)) != NVFP4_OK || (st = cache_map(&map_v, p.c.v, p.c)) != NVFP4_OK) return st;
    cudaError_t e = launch_attn(map_k, map_v, p, d->smem_optin, stream);
    return e == cudaSuccess ? NVFP4_OK : cuda_fail(e, "attention launch");
}

// Where the parts of a workspace for shared prefixes begin: the prompt kernel's
// partial results, the records, its whole results, and the chunks' parts: one a
// row and kChunkFloats more.
constexpr long long kChunkFloats = 10 << 20;
struct SharedLayout {
    size_t head, walks, records, first, rows, parts, bytes;
    long long room;  // rows of the chunks' parts
    SharedLayout(int sms, long long tokens, long long heads, long long d, long long batch) {
        size_t at = 0;
        auto take = [&](long long n) {
            const size_t here = at;
            at += ((size_t)n + 255) & ~(size_t)255;
            return here;
        };
        take((long long)attn_workspace_bytes(sms));
        head = take(sizeof(SharedHead));
        walks = take(sms * (long long)sizeof(SharedWalk));
        records = take(2 * batch * (long long)sizeof(SharedSeq));
        first = take((batch + 1) * 4);
        rows = take(tokens * heads * (d + 4) * 4);
        room = tokens * heads + kChunkFloats / (d + 4);
        parts = take(room * (d + 4) * 4);
        bytes = at;
    }
};

// Whether a call takes attention as it is, sequence by sequence (us, sequence by sequence and shared).
// Where a sequence's own rows fill half of the prompt kernel's blocks there is nothing to win: prefixes of 8192, 8 and 32
// sequences of so many rows a kv head, heads of 128: 32 rows 41 and 30, 104 and 76; 64 rows 45 and 48, 122 and 134.  Heads of
// 256: 48 rows 61 and 41, 139 and 98; 96 rows 63 and 85, 145 and 158.
// Where little is read again the plan, the join and both kernels' starts cost more, and a group's prefix itself costs the
// prompt kernel what three sequences' costs without sharing (whose later ones find it in L2).  So the prefixes of all
// sequences but three a group count: 84 MB of them 23 and 25 (8 behind 8192), 102 MB 31 and 32, 109 MB 27 and 24 (16
// behind 4096) or 33 and 29 (64, 4 groups), 123 MB 29 and 26, 134 MB 45 and 40 (5 behind 32768) or 57 and 59 (32, 8 groups),
// 167 MB 34 and 25, 201 MB 53 and 39; 67 MB, that is 4 a group: 34 and 39, 34 and 49 (4 groups), 44 and 51 (16), but 40
// and 38, 40 and 34 with heads of 256; 3 or 2 a group 32 and 39, 40 and 54.
constexpr int kSharedMostRows = 63;
constexpr long long kSharedLeastBytes = 105000000;
// Chunks of an SM, in turns (over the 14 cases that attn_shared.cu lists 41.6 us; 8: 44.0, two of them a third longer; 32: 42.2).
constexpr int kSharedItems = 16;
static bool shares_nothing(const KvBatch &n, const KvCache &c, int g, const nvfp4_kv_prefix &x, int sms) {
    if (sms > kSharedMostCtas) return true;
    if (x.groups == 0 || (long long)n.max_q * g > kSharedMostRows) return true;
    // (the plan counts in 32 bits)
    if (((long long)n.tokens * g / kPRows + x.groups) * c.heads * (n.max_kv / kPTile + kPOverShared + 1) >= kSharedMostUnits) return true;
    const long long length = n.max_kv - (x.max_own_len < n.max_kv ? x.max_own_len : n.max_kv);
    return (n.b - 3ll * x.groups) * length * c.heads * 2 * c.d < kSharedLeastBytes;
}

extern "C" nvfp4_status nvfp4_attn_paged_shared(const nvfp4_head_rows *q, const nvfp4_kv_cache *cache,
                                                const nvfp4_kv_batch *batch, const nvfp4_kv_prefix *prefix, float scale,
                                                const nvfp4_head_rows *gate, uint16_t *y, void *workspace,
                                                size_t workspace_bytes, cudaStream_t stream) {
    AttnParams p;
    nvfp4_status st = take_attn(q, cache, batch, scale, gate, y, workspace, &p);
    if (st != NVFP4_OK) return st;
    if (!prefix) return fail(NVFP4_ERR_INVALID_ARG, "null nvfp4_kv_prefix");
    if (prefix->groups < 0 || prefix->groups > batch->batch || prefix->groups > kSharedMaxGroups)
        return fail(NVFP4_ERR_INVALID_ARG, "groups = %d must be in [0, batch = %d] and at most %d", prefix->groups,
                    batch->batch, kSharedMaxGroups);
    if (prefix->groups > 0 && (!prefix->group_cu || !prefix->prefix_lens))
        return fail(NVFP4_ERR_INVALID_ARG, "prefix: null pointer");
    if (!aligned(prefix->group_cu, 4) || !aligned(prefix->prefix_lens, 4))
        return fail(NVFP4_ERR_MISALIGNED, "prefix: arrays must be 4-byte aligned");
    if (prefix->max_group_tokens < 1 || prefix->max_own_len < 0)
        return fail(NVFP4_ERR_INVALID_ARG, "prefix: max_group_tokens = %d, max_own_len = %d out of range",
                    prefix->max_group_tokens, prefix->max_own_len);
    if (p.n.b == 0) return NVFP4_OK;
    const int group_tokens = prefix->max_group_tokens < p.n.tokens ? prefix->max_group_tokens : p.n.tokens;
    if ((long long)p.n.tokens * p.q.heads > (1 << 30) || (long long)p.n.b * p.c.heads > 0x7FFFFFFF)
        return fail(NVFP4_ERR_INVALID_ARG, "tokens * heads, or batch * kv_heads, too large");
    if (!workspace) return fail(NVFP4_ERR_INVALID_ARG, "workspace: null pointer");
    int dev = 0;
    DeviceState *d = nullptr;
    if ((st = current_device(&dev, &d)) != NVFP4_OK) return st;
    const SharedLayout at(d->sms, p.n.tokens, p.q.heads, p.c.d, p.n.b);
    if (workspace_bytes < at.bytes)
        return fail(NVFP4_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed", workspace_bytes, at.bytes);
    uint8_t *const ws = static_cast<uint8_t *>(workspace);
    p.err = d->err_word;
    p.ctas = d->sms;
    p.partials = static_cast<float *>(workspace);
    p.slot_floats = kAttnSlotFloats;
    CUtensorMap map_k, map_v;
    if ((st = cache_map(&map_k, p.c.k, p.c)) != NVFP4_OK || (st = cache_map(&map_v, p.c.v, p.c)) != NVFP4_OK) return st;
    cudaError_t e;
    if (shares_nothing(p.n, p.c, p.g, *prefix, d->sms)) {
        e = launch_attn(map_k, map_v, p, d->smem_optin, stream);
        return e == cudaSuccess ? NVFP4_OK : cuda_fail(e, "attention launch");
    }
    SharedPlan plan;
    plan.n = p.n;
    plan.group_cu = prefix->group_cu;
    plan.prefix_lens = prefix->prefix_lens;
    plan.groups = prefix->groups;
    plan.max_group_tokens = group_tokens;
    plan.page_log2 = p.c.page_log2;
    plan.heads = p.c.heads;
    plan.g = p.g;
    plan.d = p.c.d;
    plan.rows_chunk = attn_chunk_rows(p.n.max_q * p.g);
    const bool eight = plan.rows_chunk == 8;
    // (over the 14 cases that attn_shared.cu lists 41.6 us; half as much 45.3, 0.7 of it 42.9, 1.4 of it 46.1, twice as much 47.3)
    plan.unit_steps = p.c.d <= 128 ? (eight ? 16.f : 9.f) : (eight ? 12.f : 8.f);
    plan.chunk_warps = attn_chunk_warps(p.c.d, eight);
    plan.of_steps = (float)p.c.heads / (d->sms * kSharedItems);
    plan.of_units = 8.f / d->sms;  // a chunk in turns may last about as long as the prompt kernel
    plan.of_rows = (float)p.c.heads * (p.c.d + 4) / (float)(kChunkFloats - (kChunkFloats >> 4));
    plan.room = (int)at.room;
    plan.head = reinterpret_cast<SharedHead *>(ws + at.head);
    plan.prefixes = reinterpret_cast<SharedSeq *>(ws + at.records);
    plan.own = plan.prefixes + plan.groups;
    plan.first = reinterpret_cast<int *>(ws + at.first);
    plan.walks = reinterpret_cast<SharedWalk *>(ws + at.walks);
    plan.ctas = p.ctas;
    plan.err = p.err;
    if ((e = launch_attn_shared_plan(plan, stream)) != cudaSuccess) return cuda_fail(e, "launch of the shared prefixes' plan");
    SharedParams pass;
    static_cast<AttnParams &>(pass) = p;
    pass.gate.p = nullptr;
    pass.n.b = prefix->groups;
    pass.n.max_q = group_tokens;
    pass.seqs = plan.prefixes;
    pass.walks = plan.walks;
    pass.rows = reinterpret_cast<float *>(ws + at.rows);
    if ((e = launch_attn_prompt_pass(map_k, map_v, pass, stream)) != cudaSuccess)
        return cuda_fail(e, "launch of attention over the shared prefixes");
    ChunkParams chunks;
    static_cast<AttnParams &>(chunks) = p;
    chunks.head = plan.head;
    chunks.own = plan.own;
    chunks.first = plan.first;
    chunks.parts = reinterpret_cast<float *>(ws + at.parts);
    chunks.room = plan.room;
    if ((e = launch_attn_chunks(chunks, stream)) != cudaSuccess) return cuda_fail(e, "attention launch");
    SharedJoin join;
    static_cast<AttnParams &>(join) = p;
    join.head = plan.head;
    join.prefixes = plan.prefixes;
    join.own = plan.own;
    join.parts = chunks.parts;
    join.rows = pass.rows;
    join.room = plan.room;
    e = launch_attn_shared_join(join, stream);
    return e == cudaSuccess ? NVFP4_OK : cuda_fail(e, "launch of the parts' join");
}

static int device_sms() {  // the GB300's where there is no device to ask
    int dev = 0, count = 0, sms = 152;
    if (cudaGetDeviceCount(&count) == cudaSuccess && count > 0 && cudaGetDevice(&dev) == cudaSuccess) {
        DeviceState *d = nullptr;
        if (device_state(dev, &d) == NVFP4_OK) sms = d->sms;
    }
    cudaGetLastError();
    return sms;
}

extern "C" nvfp4_status nvfp4_attn_shared_workspace_size(int tokens, int heads, int head_dim, int batch, size_t *bytes) {
    if (!bytes) return fail(NVFP4_ERR_INVALID_ARG, "null bytes pointer");
    nvfp4_status st = check_head_dim(head_dim);
    if (st != NVFP4_OK) return st;
    if (tokens < 0 || heads < 1 || heads > 65536 || batch < 0 || batch > 65535)
        return fail(NVFP4_ERR_INVALID_ARG, "tokens = %d, heads = %d, batch = %d (0..65535) out of range", tokens, heads, batch);
    *bytes = SharedLayout(device_sms(), tokens, heads, head_dim, batch).bytes;
    return NVFP4_OK;
}

extern "C" nvfp4_status nvfp4_attn_workspace_size(size_t *bytes) {
    if (!bytes) return fail(NVFP4_ERR_INVALID_ARG, "null bytes pointer");
    *bytes = attn_workspace_bytes(device_sms());
    return NVFP4_OK;
}
