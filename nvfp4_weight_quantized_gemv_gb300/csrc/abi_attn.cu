// abi_attn.cu -- C entry points of the attention operators: argument checks,
// workspace and launch.
#include "abi_internal.h"
#include "attn_internal.h"

#include <cmath>

namespace nvfp4 {

static bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

static nvfp4_status current_device(int *dev, DeviceState **d) {
    cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    return device_state(*dev, d);
}

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

extern "C" nvfp4_status nvfp4_attn_paged(const nvfp4_head_rows *q, const nvfp4_kv_cache *cache,
                                         const nvfp4_kv_batch *batch, float scale, const nvfp4_head_rows *gate,
                                         uint16_t *y, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    AttnParams p;
    nvfp4_status st;
    if ((st = take_cache(cache, &p.c)) != NVFP4_OK || (st = take_batch(batch, p.c, &p.n)) != NVFP4_OK) return st;
    if (!(scale > 0.f) || !std::isfinite(scale))
        return fail(NVFP4_ERR_INVALID_ARG, "scale must be positive and finite");
    if (workspace && !aligned(workspace, 256))
        return fail(NVFP4_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (p.n.b == 0) return NVFP4_OK;
    if (!q || !y) return fail(NVFP4_ERR_INVALID_ARG, "q or y: null pointer");
    if ((st = take_rows(q, "q", &p.q)) != NVFP4_OK || (st = take_rows(gate, "gate", &p.gate)) != NVFP4_OK) return st;
    if (p.q.heads % p.c.heads != 0)
        return fail(NVFP4_ERR_INVALID_ARG, "%d query heads are no multiple of %d kv heads", p.q.heads, p.c.heads);
    if (gate && p.gate.heads != p.q.heads)
        return fail(NVFP4_ERR_INVALID_ARG, "gate has %d heads, q %d", p.gate.heads, p.q.heads);
    if (!aligned(y, 16)) return fail(NVFP4_ERR_MISALIGNED, "y must be 16-byte aligned");
    if ((long long)p.n.max_q * p.q.heads > (1 << 30))
        return fail(NVFP4_ERR_INVALID_ARG, "max_q_len * heads too large");
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
    p.y = y;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.g = p.q.heads / p.c.heads;
    p.g_magic = p.g > 1 ? (unsigned)(((1ull << 32) + p.g - 1) / p.g) : 0;
    p.err = d->err_word;
    p.ctas = d->sms;
    p.partials = static_cast<float *>(workspace);
    p.slot_floats = kAttnSlotFloats;
    CUtensorMap map_k, map_v;
    if ((st = cache_map(&map_k, p.c.k, p.c)) != NVFP4_OK || (st = cache_map(&map_v, p.c.v, p.c)) != NVFP4_OK) return st;
    cudaError_t e = attn_few_rows(p.n.max_q * p.g) ? launch_attn_decode(map_k, map_v, p, d->smem_optin, stream)
                                                         : launch_attn_prompt(map_k, map_v, p, stream);
    return e == cudaSuccess ? NVFP4_OK : cuda_fail(e, "attention launch");
}

extern "C" nvfp4_status nvfp4_attn_workspace_size(size_t *bytes) {
    if (!bytes) return fail(NVFP4_ERR_INVALID_ARG, "null bytes pointer");
    int dev = 0, count = 0, sms = 152;  // the GB300's where there is no device to ask
    if (cudaGetDeviceCount(&count) == cudaSuccess && count > 0 && cudaGetDevice(&dev) == cudaSuccess) {
        DeviceState *d = nullptr;
        if (device_state(dev, &d) == NVFP4_OK) sms = d->sms;
    }
    cudaGetLastError();
    *bytes = attn_workspace_bytes(sms);
    return NVFP4_OK;
}
