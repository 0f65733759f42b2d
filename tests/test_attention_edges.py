"""Attention over the paged cache at the edges of its contract: logits far from
zero, pages of zeros, scales at their bounds, queries that are not finite,
tokens without a place.  Definitions and tolerances are those of
test_attention_ops.
"""
from __future__ import annotations

import math

import pytest
import torch

import nvfp4_weight_quantized_gemv_gb300 as nv
from test_attention_ops import Paged, attn64, built, check_attn, close_bf16, randn  # noqa: F401

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def offset_keys(p):
    """Keys whose first entry is 64 in every token, the others small: a query's first entry moves all its logits."""
    for codes in (p.k, p.v):
        codes.copy_((randn(p.g, *codes.shape) * 0.5).to(E4M3).cuda())
    p.k[..., 0] = torch.full((), 64.0).to(E4M3)


def offset_queries(p, n, hq, nats):
    q = randn(p.g, n, hq, p.d) * 1.5
    q[..., 0] = nats / (64.0 * p.d ** -0.5)
    return q.bfloat16().cuda()


# (tokens of a sequence, query heads a kv head): one row, the kernel for few rows, four copies, two, none
ROWS = [(1, 1), (3, 4), (5, 4), (20, 1), (9, 5), (40, 1), (130, 1), (70, 6)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,g", ROWS)
@pytest.mark.parametrize("nats", [-300.0, -170.0, -100.0, 250.0])
def test_logits_far_from_zero(n, g, d, nats):
    """softmax does not see an offset of all logits; a diagonal tile has whole blocks of tokens that a row does not see."""
    p = Paged(n * d, [n, n], [n + 170, n], 1, d, 32, fill=False)
    offset_keys(p)
    check_attn(p, offset_queries(p, 2 * n, g, nats))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n,g", [(5, 4), (40, 1), (70, 2)])
@pytest.mark.parametrize("nats", [-150.0, 150.0])
def test_logits_far_from_zero_in_many_sequences(n, g, d, nats):
    """So many blocks that a CTA works on several tiles of one."""
    p = Paged(n * d, [n] * 20, [n + 120 + 37 * b for b in range(20)], 8, d, 32, fill=False)
    offset_keys(p)
    check_attn(p, offset_queries(p, 20 * n, 8 * g, nats))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("n,g", ROWS)
def test_last_page_of_zeros(n, g, d, page):
    """Values that are all zero have the smallest scale there is, 2^-100."""
    p = Paged(n * d + page, [n] * 10, [n + 150] * 10, 16, d, page, fill=False)
    offset_keys(p)
    for b in range(10):
        for j in {(n + 149) // page, (n + 149) // page - 1, 1}:
            at = int(p.table[b, j])
            p.v[at], p.vs[at] = torch.zeros(()).to(E4M3), 2.0 ** -100
    check_attn(p, offset_queries(p, 10 * n, 16 * g, -40.0))


NO_PLACE = [(3, 1, 2), (4, 0, 4), (6, 2, 4), (40, 30, 1), (150, 20, 2), (20, 0, 3)]  # tokens, length with them, heads


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n,kv,g", NO_PLACE)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_query_of_a_token_without_a_place_does_not_matter(n, kv, g, d, bad):
    p = Paged(n + kv + d, [n, n], [kv, n + 60], 2, d, 32)
    q, gate = ((randn(p.g, 2 * n, 2 * g, d)).bfloat16().cuda() for _ in range(2))
    want = check_attn(p, q, gate=gate)
    assert not want[:n - kv].any()
    q[:n - kv, :, 5::7] = bad
    assert torch.equal(nv.nvfp4_attn_paged(q, *p.args(), n, n + 60, gate=gate), want)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n,kv,g", NO_PLACE)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_gate_of_a_token_without_a_place_does_not_matter(n, kv, g, d, bad):
    p = Paged(n + kv + d, [n, n], [kv, n + 60], 2, d, 32)
    q, gate = ((randn(p.g, 2 * n, 2 * g, d)).bfloat16().cuda() for _ in range(2))
    want = check_attn(p, q, gate=gate)
    gate[:n - kv, :, 3::5] = bad
    assert torch.equal(nv.nvfp4_attn_paged(q, *p.args(), n, n + 60, gate=gate), want)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n,g", [(1, 4), (4, 4), (20, 1), (40, 1), (150, 2)])
@pytest.mark.parametrize("key", [1.0, -1.0, 0.0])
def test_query_that_is_not_finite_gives_nan(n, g, d, key):
    """Whatever its scores would be: infinities of one sign, of both, or none at all."""
    p = Paged(n + d, [n], [n + 200], 1, d, 64)
    p.k[..., 3] = torch.full((), key).to(E4M3)
    q = randn(p.g, n, g, d).bfloat16().cuda()
    want = check_attn(p, q)
    q[n // 2, g - 1, 3] = math.inf
    y = nv.nvfp4_attn_paged(q, *p.args(), n, n + 200)
    assert torch.isnan(y[n // 2, g - 1]).all()
    y[n // 2, g - 1] = want[n // 2, g - 1]
    assert torch.equal(y, want)


@pytest.mark.parametrize("n,g", ROWS)
@pytest.mark.parametrize("d", [128, 256])
def test_a_large_scale_of_values_behind_tokens_of_little_weight(n, g, d):
    """One page of logits 0 and scale 1, one of logits 39 ln 2 and scale 2^100: neither the totals' nor the sums'
    units may leave the range of fp32."""
    p = Paged(n + d, [n], [n + 100], 1, d, 32, fill=False)
    p.v.copy_(randn(p.g, *p.v.shape).to(E4M3).cuda())
    at = int(p.table[0, 1])
    p.k[at, :, :, 0], p.vs[at] = torch.full((), 8.0).to(E4M3), 2.0 ** 100
    q = randn(p.g, n, g, d).bfloat16()
    q[..., 0] = 1.0
    check_attn(p, q.cuda(), scale=39 * math.log(2) / 8)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n", [2, 30, 200])
def test_rows_of_sequences_that_are_passed_over_stay_as_they_are(n, d):
    """More tokens than max_q_len, and tokens behind the last sequence's."""
    p = Paged(n + d, [n, n + 1, n], [n + 40, n + 50, n + 9], 1, d, 64)
    T = 3 * n + 1
    q = randn(p.g, T + 5, 2, d).bfloat16().cuda()
    want = nv.nvfp4_attn_paged(q[:T], *p.args(), n + 1)
    out = torch.full_like(q, 7.0)
    nv.nvfp4_attn_paged(q, *p.args(), n, out=out)
    assert nv.nvfp4_device_error() == 256
    gone = torch.zeros(T + 5, dtype=torch.bool)
    gone[n:2 * n + 1] = gone[T:] = True
    assert (out[gone.cuda()] == 7).all()
    ref, size = attn64(p, q[:T].cpu(), d ** -0.5)
    close_bf16(out[:T][~gone[:T].cuda()], ref[~gone[:T]], 2.0 ** -8 * size[~gone[:T]])
    close_bf16(want, ref, 2.0 ** -8 * size)

    k = randn(p.g, T + 5, 1, d).bfloat16().cuda()
    codes = [t.clone() for t in (p.k.view(torch.uint8), p.v.view(torch.uint8), p.ks, p.vs)]
    q_out = nv.nvfp4_kv_append(k, k, *p.args(), n, q=q, q_out=torch.full_like(q, 7.0))
    assert nv.nvfp4_device_error() == 256
    assert (q_out[gone.cuda()] == 7).all() and torch.equal(q_out[~gone.cuda()], q[~gone.cuda()])
    at = p.table[1, :-(-p.kvs[1] // 64)].long().cuda()
    for a, b in zip(codes, (p.k.view(torch.uint8), p.v.view(torch.uint8), p.ks, p.vs)):
        assert torch.equal(a[at], b[at])


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n,g", [(20, 1), (40, 1), (130, 1), (70, 6)])
def test_exponents_that_differ_by_row_and_by_block_of_tokens(n, g, d):
    """Every row has weights of its own size in every 32 tokens, up to 2^-30 of its largest and in no order."""
    p = Paged(n + d, [n, n], [n + 300, n + 20], 2, d, 32)
    block = torch.randint(-8, 9, (p.pages, 2, 1), generator=p.g).float()
    p.ks.fill_(0.125)
    p.k[..., 0] = block.to(E4M3).cuda()
    q = randn(p.g, 2 * n, 2 * g, d) * 0.1
    q[..., 0] = torch.randint(-10, 11, (2 * n, 2 * g), generator=p.g) / (8 * 0.125 * d ** -0.5)
    check_attn(p, q.bfloat16().cuda())
