"""Attention operators on the GPU against plain fp64 implementations.

  - nvfp4_qk_norm_rope: per-head RMS norm and rotation, every layout of the rows;
  - nvfp4_kv_append: codes and scales of the paged cache, byte for byte where
    no fp32 arithmetic precedes the rounding (values), to one code elsewhere;
  - nvfp4_attn_paged: softmax over the cache, from empty sequences to long ones.

Tolerances.  bf16 rounds to 2^-9 of the result, and fp32 arithmetic ahead of it
may move a value across one rounding boundary: 2^-8 |y| bounds both.  An
attention result is a weighted mean of values: weights that are held to 2^-9
(relative) add at most 2^-9 sum_j p_j |V_j|, and so does the fp32 error of a
logit (at most 2^-20 of sum |q k|, which stays below 2^9 here).
"""
from __future__ import annotations

import math

import pytest
import torch

import nvfp4_weight_quantized_gemv_gb300 as nv

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def built():
    nv.build()
    yield
    assert nv.nvfp4_device_error() == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, generator=g)


def table(positions, rot):
    half = rot // 2
    ang = torch.arange(positions, dtype=F64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=F64) / max(half, 1))
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def heads64(x, w, cs, rot, inter, eps=1e-6):
    """Norm and rotation of bf16 rows [T, H, D] in 64 bits; cs [T, rot]."""
    x = x.to(F64)
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.to(F64)
    if rot == 0:
        return x
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    c, s = cs[:, None, :rot // 2].to(F64), cs[:, None, rot // 2:].to(F64)
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def close_bf16(got, ref, extra=0.0):
    err = (got.cpu().to(F64) - ref).abs()
    lim = 2.0 ** -8 * ref.abs() + extra + 2.0 ** -100
    bad = ~(err <= lim)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} out of tolerance, worst {err[bad].max()}"


def rows(g, tokens, heads, d, layout):
    """bf16 rows [tokens, heads, d] of a larger array: contiguous, a slice of it, heads outermost, or at an odd address."""
    if layout == "slice":
        return randn(g, tokens, heads + 3, d + 8).bfloat16().cuda()[:, 2:2 + heads, 8:]
    if layout == "heads_first":
        return randn(g, heads, tokens, d).bfloat16().cuda().transpose(0, 1)
    if layout == "odd":
        return randn(g, tokens * heads * d + 1).bfloat16().cuda()[1:].view(tokens, heads, d)
    return randn(g, tokens, heads, d).bfloat16().cuda()


# ------------------------------------------------------------ norm + rotation
@pytest.mark.parametrize("tokens,hq,hk,d,rot,inter,weights,layout", [
    (1, 24, 4, 256, 64, False, True, "plain"), (5, 6, 2, 128, 128, True, True, "slice"),
    (33, 5, 1, 96, 24, False, True, "plain"), (7, 3, 3, 64, 64, False, False, "heads_first"),
    (2, 1, 1, 16, 16, True, True, "odd"), (3, 2, 1, 80, 80, False, True, "odd"), (300, 9, 0, 112, 0, False, True, "slice"),
    (4, 4, 2, 240, 18, True, False, "slice"), (6, 2, 2, 208, 100, False, True, "heads_first")])
def test_norm_rope(tokens, hq, hk, d, rot, inter, weights, layout):
    g = gen(tokens * d + rot)
    q = rows(g, tokens, hq, d, layout)
    k = rows(g, tokens, hk, d, layout) if hk else None
    qw, kw = ((1 + 0.3 * randn(g, d)).bfloat16() if weights else None for _ in range(2))
    pos = torch.randint(0, 5000, (tokens,), generator=g, dtype=torch.int32)
    cs = table(5000, rot) if rot else None
    qo, ko = nv.nvfp4_qk_norm_rope(q, k, pos.cuda() if rot else None, cs.cuda() if rot else None,
                                   q_weight=qw.cuda() if weights else None, k_weight=kw.cuda() if weights else None,
                                   interleaved=inter)
    at = cs[pos.long()] if rot else None
    close_bf16(qo, heads64(q.cpu(), qw, at, rot, inter), 2.0 ** -20)
    if hk:
        close_bf16(ko, heads64(k.cpu(), kw, at, rot, inter), 2.0 ** -20)
    else:
        assert ko is None


def test_norm_rope_in_place_and_bad_positions():
    g = gen(3)
    q = randn(g, 4, 2, 64).bfloat16().cuda()
    want, _ = nv.nvfp4_qk_norm_rope(q, None, torch.arange(4, dtype=torch.int32).cuda(), table(4, 64).cuda())
    pos = torch.tensor([0, 1, 4, -1], dtype=torch.int32).cuda()
    got, _ = nv.nvfp4_qk_norm_rope(q, None, pos, table(4, 64).cuda(), q_out=q)
    assert got.data_ptr() == q.data_ptr()
    assert torch.equal(got[:2], want[:2]) and not got[2:].any()
    assert nv.nvfp4_device_error() == 256


def test_norm_rope_of_zero_huge_and_non_finite_rows():
    x = torch.zeros(5, 1, 32).bfloat16()
    x[1], x[2], x[3, 0, 5], x[4, 0, 7] = 1e18, 1e-20, math.inf, math.nan
    w = torch.ones(32).bfloat16()
    y, _ = nv.nvfp4_qk_norm_rope(x.cuda(), None, None, None, q_weight=w.cuda())
    close_bf16(y[:3], heads64(x[:3], w, None, 0, False))
    assert torch.isnan(y[3:]).any(-1).all()


# ------------------------------------------------------------------- the cache
def need64(amax):
    """The smallest power of two s with amax <= 448 s, within 2^-100 .. 2^100."""
    _, e = torch.frexp(amax.to(F64))
    s = 2.0 ** (e.to(F64) - 10)
    for _ in range(3):
        s = torch.where(amax > 448 * s, 2 * s, s)
    return torch.where(amax > 0, s, torch.full_like(s, 0.0)).clamp(2.0 ** -100, 2.0 ** 100)


def e4m3_64(x):
    """Nearest E4M3 value, ties to even, saturated; an infinity or NaN is NaN."""
    _, e = torch.frexp(x)
    step = 2.0 ** (e.to(F64) - 4).clamp(min=-9)
    y = (torch.round(x / step) * step).clamp(-448, 448)
    return torch.where(torch.isfinite(x), y, torch.full_like(x, math.nan))


class Paged:
    """A cache, a batch over it and their copies for the fp64 side."""

    def __init__(self, seed, qs, kvs, hkv, d, page, layout="plain", fill=True, spare=2):
        g = self.g = gen(seed)
        self.qs, self.kvs, self.hkv, self.d, self.page = qs, kvs, hkv, d, page
        need = [-(-kv // page) for kv in kvs]
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=g)
        self.table = torch.full((len(qs), max(need + [1]) + 1), 1 << 30, dtype=torch.int32)  # never to be read
        n = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[n:n + k]
            n += k
        self.cu = torch.tensor([sum(qs[:i]) for i in range(len(qs) + 1)], dtype=torch.int32)
        shape = (self.pages, hkv, page, d)
        if layout == "plain":
            k, v = torch.zeros(shape, dtype=torch.uint8).cuda(), torch.zeros(shape, dtype=torch.uint8).cuda()
        elif layout == "tokens_first":  # [pages, 2, page, heads, d]
            both = torch.zeros((self.pages, 2, page, hkv, d), dtype=torch.uint8).cuda()
            k, v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
        else:  # "padded": a wider array
            both = torch.zeros((2, hkv, self.pages, page, d + 32), dtype=torch.uint8).cuda()
            k, v = both[0].transpose(0, 1)[..., 16:16 + d], both[1].transpose(0, 1)[..., 16:16 + d]
        self.k, self.v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
        self.ks, self.vs = torch.ones(self.pages, hkv).cuda(), torch.ones(self.pages, hkv).cuda()
        if fill:
            for codes, scale in ((self.k, self.ks), (self.v, self.vs)):
                x = randn(g, *shape)
                s = 2.0 ** torch.randint(-12, 0, (self.pages, hkv), generator=g)
                codes.copy_(e4m3_64(x.to(F64) * 32).float().to(torch.float8_e4m3fn).cuda())
                scale.copy_(s.cuda() / 8)
        self.dev = [t.cuda() for t in (self.table, self.cu, torch.tensor(kvs, dtype=torch.int32))]

    def host(self):
        return [t.cpu().to(F64) if t.dtype == torch.float32 else t.cpu().float().to(F64)
                for t in (self.k, self.v, self.ks, self.vs)]

    def args(self):
        return (self.k, self.v, self.ks, self.vs, *self.dev)


def append64(p, k64, v64, k, v, ks, vs):
    """The header's definition of an append, on the fp64 copies, in place."""
    for codes, scales, new in ((k, ks, k64), (v, vs, v64)):
        for b, (q, kv) in enumerate(zip(p.qs, p.kvs)):
            start, t0 = kv - q, int(p.cu[b])
            for pg in range(max(start, 0) // p.page, -(-kv // p.page)):
                lo, hi = max(start, 0, pg * p.page), min(kv, (pg + 1) * p.page)
                x = new[t0 + lo - start:t0 + hi - start].transpose(0, 1)  # [H, n, D]
                page, base = int(p.table[b, pg]), pg * p.page
                fin = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
                s = need64(fin.amax((1, 2)))
                if lo > base:
                    s = torch.maximum(s, scales[page])
                    codes[page, :, :lo - base] = e4m3_64(codes[page, :, :lo - base] * (scales[page] / s)[:, None, None])
                scales[page] = s
                codes[page, :, lo - base:hi - base] = e4m3_64(x / s[:, None, None])


def same_codes(got, ref, exact):
    got = got.cpu().float().to(F64)
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    diff = torch.nan_to_num(got - ref, 0.0).abs()
    if exact:
        assert not diff.any()
        return
    # a value within 2^-20 of a rounding boundary may take the neighbouring code
    step = 2.0 ** (torch.frexp(ref)[1].to(F64) - 4).clamp(min=-9)
    assert (diff <= step).all()
    assert (diff > 0).double().mean() < 1e-3


@pytest.mark.parametrize("qs,kvs,hq,hkv,d,page,rot,inter,weights,layout,rlayout", [
    ([1, 1, 1], [1, 40, 65], 6, 2, 256, 64, 64, False, True, "plain", "slice"),
    ([1], [17], 0, 1, 128, 16, 128, True, True, "tokens_first", "plain"),
    ([2, 2], [33, 2], 4, 4, 64, 32, 64, False, True, "padded", "heads_first"),
    ([5, 0, 130, 3], [5, 0, 200, 66], 3, 1, 96, 64, 24, False, True, "plain", "odd"),
    ([37, 300], [1000, 300], 8, 2, 128, 16, 0, False, False, "tokens_first", "slice"),
    ([257], [257], 2, 2, 256, 256, 256, True, True, "padded", "plain"),
    ([1, 4], [0, 2], 2, 1, 32, 16, 32, False, False, "plain", "plain"),   # tokens without a place
    ([600], [700], 1, 1, 16, 128, 4, False, True, "plain", "plain")])
def test_append(qs, kvs, hq, hkv, d, page, rot, inter, weights, layout, rlayout):
    p = Paged(sum(qs) + d, qs, kvs, hkv, d, page, layout)
    g, T = p.g, sum(qs)
    q = rows(g, T, hq, d, rlayout) if hq else None
    k, v = rows(g, T, hkv, d, rlayout), rows(g, T, hkv, d, rlayout)
    qw, kw = ((1 + 0.3 * randn(g, d)).bfloat16() if weights else None for _ in range(2))
    cs = table(max(kvs) + 3, rot) if rot else None
    ref = p.host()
    qo = nv.nvfp4_kv_append(k, v, *p.args(), max(qs), cos_sin=cs.cuda() if rot else None,
                            k_weight=kw.cuda() if weights else None, q=q, q_weight=qw.cuda() if weights else None,
                            interleaved=inter)
    pos = torch.cat([torch.arange(kv - n, kv) for n, kv in zip(qs, kvs)])
    at = cs[pos.clamp(min=0)] if rot else None
    append64(p, heads64(k.cpu(), kw, at, rot, inter), v.cpu().to(F64), *ref)
    assert torch.equal(p.vs.cpu().to(F64), ref[3]) and torch.equal(p.ks.cpu().to(F64), ref[2])
    same_codes(p.v, ref[1], True)
    same_codes(p.k, ref[0], not weights and not rot)
    if hq:
        want = heads64(q.cpu(), qw, at, rot, inter)
        want[pos < 0] = 0
        close_bf16(qo, want, 2.0 ** -20)
    else:
        assert qo is None


def test_append_one_by_one_grows_the_scale():
    """Tokens that get larger: every append rewrites the page for the larger scale, as the definition says."""
    p = Paged(5, [1], [1], 2, 64, 16, fill=False, spare=4)
    ref = p.host()
    for n in range(1, 17):
        p.kvs, kv = [n], torch.tensor([n], dtype=torch.int32).cuda()
        x = (randn(p.g, 1, 2, 64) * 3.0 ** n).bfloat16()
        nv.nvfp4_kv_append(x.cuda(), (-x).cuda(), p.k, p.v, p.ks, p.vs, p.dev[0], p.dev[1], kv, 1)
        append64(p, x.to(F64), -x.to(F64), *ref)
        assert torch.equal(p.ks.cpu().to(F64), ref[2])
        same_codes(p.k, ref[0], True)
        same_codes(p.v, ref[1], True)


def test_append_extremes():
    p = Paged(6, [6], [6], 1, 32, 16, fill=False)
    x = torch.ones(6, 1, 32).bfloat16()
    x[0], x[1, 0, 3], x[2, 0, 4], x[3, 0, 5], x[4], x[5] = 0, math.inf, -math.inf, math.nan, 1e-30, 1000
    ref = p.host()
    nv.nvfp4_kv_append(x.cuda(), x.cuda(), *p.args(), 6)
    append64(p, x.to(F64), x.to(F64), *ref)
    assert torch.equal(p.ks.cpu().to(F64), ref[2])
    same_codes(p.k, ref[0], True)
    # nothing but zeros, and values whose scale meets its bounds
    for val, want in ((0.0, 2.0 ** -100), (1e-38, 2.0 ** -100), (3e38, 2.0 ** 100)):
        p = Paged(7, [1], [1], 1, 16, 16, fill=False)
        y = torch.full((1, 1, 16), val).bfloat16().cuda()
        nv.nvfp4_kv_append(y, y, *p.args(), 1)
        assert float(p.ks[int(p.table[0, 0]), 0]) == want
        assert float(p.k[int(p.table[0, 0]), 0, 0, 0].float()) == (448.0 if val > 1 else 0.0)


def test_append_ignores_bad_paging_data():
    p = Paged(8, [2, 2], [10, 10], 1, 32, 16)
    before = [t.clone().view(torch.uint8) if t.dtype != torch.float32 else t.clone() for t in (p.k, p.v, p.ks, p.vs)]
    x = randn(p.g, 4, 1, 32).bfloat16().cuda()
    t = p.dev[0].clone()
    t[0, 0], t[1, 0] = p.pages, -1
    nv.nvfp4_kv_append(x, x, p.k, p.v, p.ks, p.vs, t, p.dev[1], p.dev[2], 2)
    assert nv.nvfp4_device_error() == 256
    for cu in ([0, 3, 2], [0, 4, 5], [-1, 0, 1]):
        c = torch.tensor(cu, dtype=torch.int32).cuda()
        nv.nvfp4_kv_append(x, x, p.k, p.v, p.ks, p.vs, t, c, torch.tensor([0, -5], dtype=torch.int32).cuda(), 2)
        assert nv.nvfp4_device_error() == 256
    for a, b in zip(before, (p.k, p.v, p.ks, p.vs)):
        assert torch.equal(a, b.view(torch.uint8) if b.dtype != torch.float32 else b)


# ------------------------------------------------------------------- attention
def attn64(p, q, scale, gate=None):
    """(y, sum_j p_j |V_j|) of every row in 64 bits."""
    kc, vc, ks, vs = p.host()
    T, hq, d = q.shape
    y, size = torch.zeros(T, hq, d, dtype=F64), torch.zeros(T, hq, d, dtype=F64)
    for b, (n, kv) in enumerate(zip(p.qs, p.kvs)):
        t0, np_ = int(p.cu[b]), -(-kv // p.page)
        if n == 0 or kv == 0:
            continue
        at = p.table[b, :np_].long()
        k, v = ((c[at] * s[at][:, :, None, None]).transpose(0, 1).reshape(p.hkv, -1, p.d)[:, :kv]
                for c, s in ((kc, ks), (vc, vs)))
        pos = torch.arange(kv - n, kv)
        hidden = torch.arange(kv) > pos[:, None]
        for h in range(hq):
            kh, vh = k[h // (hq // p.hkv)], v[h // (hq // p.hkv)]
            s = (q[t0:t0 + n, h].to(F64) @ kh.T * scale).masked_fill(hidden, -math.inf)
            w = torch.softmax(s, -1)
            w[pos < 0] = 0
            y[t0:t0 + n, h], size[t0:t0 + n, h] = w @ vh, w @ vh.abs()
    if gate is not None:
        z = torch.sigmoid(gate.to(F64))
        y, size = y * z, size * z
    return y, size


def check_attn(p, q, gate=None, scale=None, **kw):
    y = nv.nvfp4_attn_paged(q, *p.args(), max(p.qs), kw.pop("max_kv", max(max(p.kvs), 1)), scale=scale, gate=gate, **kw)
    ref, size = attn64(p, q.cpu(), p.d ** -0.5 if scale is None else scale, None if gate is None else gate.cpu())
    close_bf16(y, ref, 2.0 ** -8 * size)
    assert nv.nvfp4_device_error() == 0
    return y


@pytest.mark.parametrize("qs,kvs,g,hkv,d,page,layout", [
    ([1], [1], 1, 1, 128, 16, "plain"), ([1], [2], 4, 2, 64, 16, "plain"), ([1, 1, 1], [300, 7, 64], 6, 4, 256, 64, "plain"),
    ([1] * 9, [1, 15, 16, 17, 63, 64, 65, 129, 500], 8, 1, 128, 32, "tokens_first"),
    ([1, 1], [1000, 0], 7, 2, 96, 128, "padded"), ([1, 1], [513, 2000], 16, 1, 128, 256, "plain"),
    ([1], [5000], 12, 1, 256, 64, "tokens_first"), ([1, 1], [260, 130], 1, 3, 16, 16, "plain"),
    ([1, 1], [700, 90], 5, 2, 208, 64, "padded"), ([1] * 40, list(range(1, 4000, 100)), 2, 1, 80, 64, "plain")])
def test_attn_decode(qs, kvs, g, hkv, d, page, layout):
    p = Paged(sum(kvs) + d, qs, kvs, hkv, d, page, layout)
    q = (randn(p.g, sum(qs), g * hkv, d) * 1.5).bfloat16().cuda()
    check_attn(p, q)


@pytest.mark.parametrize("qs,kvs,g,hkv,d,page", [
    ([5, 2, 8], [100, 2, 513], 5, 2, 128, 64), ([3, 0, 4], [3, 0, 777], 8, 1, 256, 16), ([4, 7], [2, 3], 3, 1, 64, 16),
    ([130], [130], 1, 2, 128, 32), ([33, 100], [400, 129], 6, 1, 256, 64), ([257, 1, 20], [900, 900, 20], 4, 2, 96, 128),
    ([128], [128], 1, 1, 64, 64), ([400], [1400], 8, 1, 128, 256), ([65, 3], [64, 1], 2, 1, 160, 16),
    ([1000], [1000], 3, 1, 128, 64), ([17] * 12, list(range(20, 1000, 83)), 2, 2, 128, 32), ([300], [2000], 12, 1, 256, 128)])
def test_attn_several_tokens(qs, kvs, g, hkv, d, page):
    p = Paged(sum(kvs) + d, qs, kvs, hkv, d, page)
    q = (randn(p.g, sum(qs), g * hkv, d) * 1.5).bfloat16().cuda()
    gate = randn(p.g, sum(qs), g * hkv, d).bfloat16().cuda()
    check_attn(p, q, gate=gate)


@pytest.mark.parametrize("n,kv", [(1, 200), (6, 90), (150, 333)])
@pytest.mark.parametrize("layout", ["slice", "heads_first", "odd"])
def test_attn_row_layouts_and_scale(n, kv, layout):
    p = Paged(n + kv, [n, 1], [kv, 50], 2, 128, 16)
    q, gate = rows(p.g, n + 1, 6, 128, layout), rows(p.g, n + 1, 6, 128, layout)
    check_attn(p, q, gate=gate, scale=0.2, max_kv=None)


@pytest.mark.parametrize("n,d", [(1, 128), (1, 256), (9, 128), (200, 128), (200, 256)])
def test_attn_slots_nobody_sees_hold_nan(n, d):
    """Slots behind the last token, pages of nobody, and whatever their scales are."""
    p = Paged(n + d, [n, n], [n + 70, n + 5], 2, d, 64)
    used = torch.zeros(p.pages, p.page, dtype=torch.bool)
    for b, kv in enumerate(p.kvs):
        for j in range(kv):
            used[int(p.table[b, j // p.page]), j % p.page] = True
    for codes in (p.k, p.v):
        raw = codes.view(torch.uint8)
        raw.copy_(torch.where(used[:, None, :, None].cuda(), raw, torch.full_like(raw, 0x7F)))
    empty = ~used.any(1)
    p.ks[empty.cuda()], p.vs[empty.cuda()] = math.nan, math.inf
    host = p.host
    p.host = lambda: [torch.nan_to_num(t, 0.0, 1.0) for t in host()]
    q = (randn(p.g, 2 * n, 4, d) * 1.5).bfloat16().cuda()
    check_attn(p, q)


@pytest.mark.parametrize("n,d", [(5, 128), (20, 256), (140, 128), (140, 256)])
def test_attn_nan_reaches_only_rows_that_see_it(n, d):
    p = Paged(n * d, [n], [n + 30], 1, d, 32)
    q = (randn(p.g, n, 3, d)).bfloat16().cuda()
    y = check_attn(p, q)
    j = 30 + n // 2  # position of token n // 2
    page, slot = int(p.table[0, j // 32]), j % 32
    v = p.v.view(torch.uint8)
    v[page, 0, slot, 7] = 0x7F
    z = nv.nvfp4_attn_paged(q, *p.args(), n, n + 30)
    assert torch.equal(z[:n // 2], y[:n // 2])
    assert torch.isnan(z[n // 2:, :, 7]).all()
    rest = torch.cat([z[n // 2:, :, :7], z[n // 2:, :, 8:]], -1)
    assert torch.equal(rest, torch.cat([y[n // 2:, :, :7], y[n // 2:, :, 8:]], -1))
    v[page, 0, slot, 7] = 0
    p.k.view(torch.uint8)[page, 0, slot, 9] = 0xFF
    z = nv.nvfp4_attn_paged(q, *p.args(), n, n + 30)
    assert torch.equal(z[:n // 2], y[:n // 2]) and torch.isnan(z[n // 2:]).all()


@pytest.mark.parametrize("n,kv,d", [(1, 3000, 128), (1, 900, 256), (4, 2500, 128), (130, 2000, 128), (130, 1000, 256)])
def test_attn_one_token_against_a_crowd(n, kv, d):
    """One logit far above all others, whose weights add up to as much: none of them may be lost."""
    p = Paged(kv, [n], [kv], 1, d, 64, fill=False)
    for codes in (p.k, p.v):
        codes.copy_((randn(p.g, *codes.shape).sign() * 0.5).to(torch.float8_e4m3fn).cuda())
    p.v[..., :d // 2] = p.v[..., :d // 2].float().abs().to(torch.float8_e4m3fn)
    p.k[int(p.table[0, 0]), 0, 5] = torch.full((d,), 8.0).to(torch.float8_e4m3fn)
    p.v[int(p.table[0, 0]), 0, 5] = (-p.v[int(p.table[0, 0]), 0, 5].float()).to(torch.float8_e4m3fn)
    q = torch.full((n, 2, d), 1.0).bfloat16().cuda()
    check_attn(p, q, scale=math.log(kv) / (8.0 * d))


@pytest.mark.parametrize("n", [1, 3, 150])
def test_attn_scales_and_queries_of_any_size(n):
    d = 128
    p = Paged(n + 1, [n], [n + 400], 2, d, 16)
    p.vs.copy_((2.0 ** torch.randint(-90, 90, p.vs.shape, generator=p.g).float()).cuda())
    p.ks.mul_(1.37)
    q = (randn(p.g, n, 4, d) * 2.0 ** torch.randint(-30, 2, (n, 4, 1), generator=p.g)).bfloat16().cuda()
    check_attn(p, q)
    p.ks.mul_(2.0 ** -60)
    q = (randn(p.g, n, 4, d) * 2.0 ** 60).bfloat16().cuda()
    check_attn(p, q)


def test_attn_bad_paging_data_reads_as_zeros():
    p = Paged(11, [1, 1], [100, 100], 1, 64, 16)
    q = randn(p.g, 2, 2, 64).bfloat16().cuda()
    good = nv.nvfp4_attn_paged(q, *p.args(), 1, 100)
    t = p.dev[0].clone()
    t[1, 2], t[1, 3] = p.pages, -7
    y = nv.nvfp4_attn_paged(q, *p.args()[:4], t, *p.dev[1:], 1, 100)
    assert nv.nvfp4_device_error() == 256
    assert torch.equal(y[0], good[0]) and torch.isfinite(y).all()
    y = nv.nvfp4_attn_paged(q, *p.args()[:6], torch.tensor([100, 101], dtype=torch.int32).cuda(), 1, 100)
    assert nv.nvfp4_device_error() == 256
    assert torch.equal(y[0], good[0]) and not y[1].any()


@pytest.mark.parametrize("qs,kvs,d", [([1] * 5, [9000, 30, 1, 4000, 700], 256), ([4, 1], [3000, 800], 128),
                                      ([200, 64], [1200, 900], 128)])
def test_attn_same_bits_every_time_and_on_other_streams(qs, kvs, d):
    p = Paged(sum(kvs), qs, kvs, 2, d, 64)
    q = randn(p.g, sum(qs), 8, d).bfloat16().cuda()
    y = nv.nvfp4_attn_paged(q, *p.args(), max(qs), max(kvs))
    ws = torch.zeros(nv.nvfp4_attn_workspace_size(), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(s):
            a = nv.nvfp4_attn_paged(q, *p.args(), max(qs), max(kvs))
            b = nv.nvfp4_attn_paged(q, *p.args(), max(qs), max(kvs), workspace=ws)
        c = nv.nvfp4_attn_paged(q, *p.args(), max(qs), max(kvs))
        torch.cuda.synchronize()
        assert torch.equal(a, y) and torch.equal(b, y) and torch.equal(c, y)


def test_append_and_attend_in_a_captured_graph():
    """One captured decode step, replayed as the sequences grow."""
    p = Paged(21, [1, 1], [40, 200], 2, 128, 16, spare=0)
    table_, kv = p.dev[0].clone(), torch.tensor([30, 190], dtype=torch.int32).cuda()
    x = randn(p.g, 2, 8, 128).bfloat16().cuda()
    cs = table(256, 128).cuda()

    def step():
        q = nv.nvfp4_kv_append(x[:, 4:6], x[:, 6:], p.k, p.v, p.ks, p.vs, table_, p.dev[1], kv, 1, cos_sin=cs, q=x[:, :4])
        return nv.nvfp4_attn_paged(q, p.k, p.v, p.ks, p.vs, table_, p.dev[1], kv, 1, 200)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y = step()
    for n in range(10):
        x.copy_(randn(p.g, 2, 8, 128).bfloat16())
        kv.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        p.kvs = kv.tolist()
        q = nv.nvfp4_qk_norm_rope(x[:, :4], None, kv - 1, cs)[0]
        ref, size = attn64(p, q.cpu(), 128 ** -0.5)
        close_bf16(y, ref, 2.0 ** -8 * size)


def test_empty_calls_do_nothing():
    p = Paged(1, [0], [5], 1, 32, 16)
    q = torch.empty((0, 2, 32), dtype=torch.bfloat16, device="cuda")
    k = torch.empty((0, 1, 32), dtype=torch.bfloat16, device="cuda")
    assert nv.nvfp4_attn_paged(q, *p.args(), 1, 5).shape == (0, 2, 32)
    assert nv.nvfp4_kv_append(k, k, *p.args(), 1, q=q).shape == (0, 2, 32)
    assert nv.nvfp4_qk_norm_rope(q, k, None, None)[0].shape == (0, 2, 32)
