"""Attention operators where the work is split: long caches over many CTAs and
ring buffers that wrap, blocks joined from parts, sizes on both sides of each
choice of kernel.  Definitions and tolerances are those of test_attention_ops.
"""
from __future__ import annotations

import pytest
import torch

import nvfp4_weight_quantized_gemv_gb300 as nv
from test_attention_ops import (F64, Paged, append64, built, check_attn, close_bf16, gen, heads64, randn,  # noqa: F401
                                rows, same_codes, table)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("qs,kvs,g,hkv,d,page", [
    ([1], [90001], 8, 1, 128, 64),                  # eight rows, two rings' worth of tiles a CTA and more
    ([2], [70000], 8, 1, 96, 16),                   # sixteen rows, pages that end inside a tile
    ([1, 1], [60003, 21], 6, 1, 256, 64),
    ([2], [50000], 8, 1, 256, 128),
    ([3], [60001], 8, 1, 128, 64),                  # 24 rows: the kernel for prompts
    ([1] * 90, [1 + 97 * (i % 23) for i in range(90)], 4, 2, 128, 32)])  # more blocks than CTAs
def test_attn_long_ranges_and_the_same_every_time(qs, kvs, g, hkv, d, page):
    p = Paged(sum(kvs) + d, qs, kvs, hkv, d, page)
    q = (randn(p.g, sum(qs), g * hkv, d) * 1.5).bfloat16().cuda()
    y = check_attn(p, q)
    for _ in range(20):
        assert torch.equal(nv.nvfp4_attn_paged(q, *p.args(), max(qs), max(kvs)), y)


def test_attn_parts_of_an_earlier_call_are_not_met_again():
    """Sequences that bring no token, after a call in which they had one; lengths of zero and one beside long ones."""
    p = Paged(31, [1, 1, 1, 1, 1], [5000, 4000, 3000, 2, 1], 2, 128, 64)
    q = (randn(p.g, 5, 8, 128) * 1.5).bfloat16().cuda()
    check_attn(p, q)
    for qs, kvs in (([2, 0, 1, 0, 1], [5000, 4000, 0, 2, 1]), ([0, 0, 0, 0, 1], [5000, 4000, 3000, 2, 1]),
                    ([1, 1, 0, 1, 2], [17, 4000, 3000, 1, 1])):
        p.qs, p.kvs = qs, kvs
        p.cu = torch.tensor([sum(qs[:i]) for i in range(6)], dtype=torch.int32)
        p.dev[1:] = [p.cu.cuda(), torch.tensor(kvs, dtype=torch.int32).cuda()]
        q = (randn(p.g, sum(qs), 8, 128) * 1.5).bfloat16().cuda()
        check_attn(p, q, max_kv=5000)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("kv", [511, 512, 513, 1023, 1024, 1025, 2049])
def test_attn_around_the_length_that_one_cta_reads(d, kv):
    p = Paged(kv + d, [1, 1], [kv, kv // 2], 3, d, 64)
    q = (randn(p.g, 2, 12, d) * 1.5).bfloat16().cuda()
    check_attn(p, q)
    check_attn(p, q, max_kv=None)  # what the table could hold


@pytest.mark.parametrize("b,hkv,g,d,longest", [(67, 8, 4, 128, 34), (40, 4, 8, 256, 300), (300, 1, 12, 96, 600), (39, 4, 2, 64, 640)])
def test_attn_many_short_blocks(b, hkv, g, d, longest):
    p = Paged(b + d, [int(i % 7 != 3) for i in range(b)], [1 + (i * 37) % longest for i in range(b)], hkv, d, 32)
    q = (randn(p.g, sum(p.qs), hkv * g, d) * 1.5).bfloat16().cuda()
    gate = randn(p.g, sum(p.qs), hkv * g, d).bfloat16().cuda()
    check_attn(p, q, gate=gate, max_kv=longest)


@pytest.mark.parametrize("n,g,d,kv", [(17, 1, 128, 300), (5, 5, 128, 3000), (8, 4, 256, 900), (33, 1, 256, 333), (8, 8, 128, 2500),
                                      (7, 7, 64, 1200), (16, 4, 96, 64), (13, 5, 256, 5000)])
@pytest.mark.parametrize("gated", [False, True])
def test_attn_rows_in_copies(n, g, d, kv, gated):
    """17 to 65 query rows a kv head, blocks of one CTA and of several, sequences that bring fewer and no tokens."""
    p = Paged(n * g + kv, [n, 1, 0, n - 3, n], [kv, 40, 30, max(n, kv // 3), n], 2, d, 64)
    q = (randn(p.g, sum(p.qs), 2 * g, d) * 1.5).bfloat16().cuda()
    gate = randn(p.g, sum(p.qs), 2 * g, d).bfloat16().cuda() if gated else None
    check_attn(p, q, gate=gate)


def test_attn_scales_of_parts_far_apart():
    """Pages whose scales differ by 2^80 in different parts of one block."""
    p = Paged(41, [1], [40000], 1, 128, 64)
    s = torch.ones(p.pages, 1)
    at = p.table[0, :40000 // 64].long()
    s[at[:200]], s[at[200:400]] = 2.0 ** -60, 2.0 ** 20
    p.vs.copy_(s.cuda())
    check_attn(p, (randn(p.g, 1, 8, 128) * 1.5).bfloat16().cuda())


@pytest.mark.parametrize("tokens,hq,hk,d,rot,inter,weights,layout", [
    (5000, 6, 1, 64, 64, False, True, "plain"), (4003, 5, 2, 128, 128, True, True, "heads_first"),
    (2111, 7, 1, 256, 64, False, True, "slice"), (2001, 6, 3, 96, 24, False, True, "plain"),
    (3001, 5, 1, 80, 20, False, False, "odd"), (2500, 9, 0, 208, 0, False, True, "plain")])
def test_norm_rope_of_many_tokens(tokens, hq, hk, d, rot, inter, weights, layout):
    g = gen(tokens + d)
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


def test_norm_rope_of_many_tokens_with_bad_positions():
    g = gen(9)
    q = randn(g, 3000, 8, 128).bfloat16().cuda()
    pos = torch.arange(3000, dtype=torch.int32)
    pos[7], pos[2999] = -1, 3000
    got, _ = nv.nvfp4_qk_norm_rope(q, None, pos.cuda(), table(3000, 64).cuda())
    pos[7] = pos[2999] = 0
    want, _ = nv.nvfp4_qk_norm_rope(q, None, pos.cuda(), table(3000, 64).cuda())
    want[7] = want[2999] = 0
    assert torch.equal(got, want)
    assert nv.nvfp4_device_error() == 256


@pytest.mark.parametrize("qs,kvs,hq,hkv,d,page,rot,inter,layout", [
    ([700], [900], 5, 2, 256, 256, 64, False, "plain"),   # pages whose values do not fit shared memory
    ([700], [900], 5, 2, 256, 64, 64, False, "heads_first"), ([3, 260, 64], [40, 300, 64], 6, 2, 128, 128, 128, True, "plain"),
    ([2] * 20, list(range(2, 402, 20)), 9, 3, 256, 16, 256, False, "plain"),
    ([5] * 7, [5, 16, 17, 18, 19, 20, 21], 2, 1, 64, 16, 32, True, "odd"), ([1000], [1000], 1, 1, 48, 32, 20, False, "plain")])
def test_append_many_tokens(qs, kvs, hq, hkv, d, page, rot, inter, layout):
    p = Paged(sum(qs) + d, qs, kvs, hkv, d, page)
    g, T = p.g, sum(qs)
    q, k, v = rows(g, T, hq, d, layout), rows(g, T, hkv, d, layout), rows(g, T, hkv, d, layout)
    qw, kw = ((1 + 0.3 * randn(g, d)).bfloat16() for _ in range(2))
    cs = table(max(kvs), rot)
    ref = p.host()
    qo = nv.nvfp4_kv_append(k, v, *p.args(), max(qs), cos_sin=cs.cuda(), k_weight=kw.cuda(), q=q, q_weight=qw.cuda(),
                            interleaved=inter)
    at = cs[torch.cat([torch.arange(kv - n, kv) for n, kv in zip(qs, kvs)])]
    append64(p, heads64(k.cpu(), kw, at, rot, inter), v.cpu().to(F64), *ref)
    assert torch.equal(p.vs.cpu().to(F64), ref[3]) and torch.equal(p.ks.cpu().to(F64), ref[2])
    same_codes(p.v, ref[1], True)
    same_codes(p.k, ref[0], False)
    close_bf16(qo, heads64(q.cpu(), qw, at, rot, inter), 2.0 ** -20)


def test_norm_rope_in_place_with_pairs_in_any_lane():
    g = gen(11)
    q = randn(g, 700, 3, 80).bfloat16().cuda()
    pos = torch.randint(0, 900, (700,), generator=g, dtype=torch.int32).cuda()
    w = (1 + 0.3 * randn(g, 80)).bfloat16().cuda()
    want, _ = nv.nvfp4_qk_norm_rope(q, None, pos, table(900, 20).cuda(), q_weight=w)
    got, _ = nv.nvfp4_qk_norm_rope(q, None, pos, table(900, 20).cuda(), q_weight=w, q_out=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)


def test_example_decodes(capsys):
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import decode_attention
    err, y = decode_attention.main(["--batch", "3", "--prompt", "90", "--steps", "5"])
    assert err < 2.0 ** -7 and y.shape == (3, 5120) and torch.isfinite(y).all()
    assert "us a step" in capsys.readouterr().out


@pytest.mark.parametrize("n,d,kv", [(1, 256, 700), (1, 128, 5000), (5, 128, 900), (40, 128, 900)])
def test_calls_in_a_row_need_no_synchronisation(n, d, kv):
    """Projection, append, norm and attention, each on what the call just ahead wrote, bit for bit as with waits between."""
    g = gen(kv + n)
    hq, hkv, b = 8, 2, 3
    w = (torch.randn(3 * hq * d, 512, generator=g) * 0.05).bfloat16().cuda()
    w4 = nv.nvfp4_quantize_bf16(w)
    cs, weight = table(kv + 16 * n, 64).cuda(), (1 + 0.3 * randn(g, d)).bfloat16().cuda()
    x = randn(g, 12, b * n, 512).bfloat16().cuda()

    def run(wait):
        p = Paged(7, [n] * b, [kv + 12 * n] * b, hkv, d, 64)
        lens = torch.full((b,), kv, dtype=torch.int32, device="cuda")
        ys = []
        for step in range(12):
            lens += n
            rows_ = nv.nvfp4_gemv_batched(*w4, x[step]).unflatten(1, (3 * hq, d))
            wait()
            q = nv.nvfp4_kv_append(rows_[:, :hkv], rows_[:, hkv:2 * hkv], p.k, p.v, p.ks, p.vs, p.dev[0], p.dev[1], lens, n,
                                   cos_sin=cs, k_weight=weight, q=rows_[:, hq:2 * hq], q_weight=weight)
            wait()
            y = nv.nvfp4_attn_paged(q, p.k, p.v, p.ks, p.vs, p.dev[0], p.dev[1], lens, n, gate=rows_[:, 2 * hq:])
            wait()
            z, _ = nv.nvfp4_qk_norm_rope(y, None, None, None, q_weight=weight)
            wait()
            ys += [q, y, z]
        torch.cuda.synchronize()
        return ys + [p.ks, p.vs, p.k.view(torch.uint8), p.v.view(torch.uint8)]

    want = run(torch.cuda.synchronize)
    for _ in range(3):
        for a, c in zip(run(lambda: None), want):
            assert torch.equal(a, c)
