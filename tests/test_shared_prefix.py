"""Attention for batches that share prefixes, against attention over each sequence's whole table in 64 bits.

A call shares only what can be worth it: 105 MB in the prefixes of all sequences but three a group, as far as
max_kv_len tells, for sequences of fewer than 64 query rows a kv head.  The tables here are wide enough for short prefixes
to be shared, and sequences that hold and bring nothing make up for groups of fewer than four.

The tolerances are those of attention over the paged cache: weights held to 2^-9, the result's rounding to bf16, fp32
logits.  Joining the two passes adds a weight's fp32 error to either side's result: 2^-20 of it, far below.
"""
from __future__ import annotations

import math

import pytest
import torch

import nvfp4_weight_quantized_gemv_gb300 as nv
from test_attention_ops import Paged, attn64, built, close_bf16, randn, rows  # noqa: F401

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Shared(Paged):
    """A paged batch whose groups' first tokens lie in the pages of the group's first sequence."""

    def __init__(self, seed, qs, kvs, groups, prefixes, hkv, d, page, **kw):
        more = max(0, 3 * len(prefixes) + 1 - len(qs))
        qs, kvs = qs + [0] * more, kvs + [0] * more
        super().__init__(seed, qs, kvs, hkv, d, page, **kw)
        self.group_cu, self.prefixes = groups, prefixes
        for g, n in enumerate(prefixes):
            for b in range(groups[g], groups[g + 1]):
                k = min(n, max(kvs[b], 0)) // page
                first = max(range(groups[g], groups[g + 1]), key=lambda i: kvs[i])  # it holds the whole prefix
                self.table[b, :k] = self.table[first, :k]
        # columns that nobody reads, for a bound on the lengths that allows for 105 MB
        columns = -(-110_000_000 // ((len(qs) - 3 * len(prefixes)) * hkv * 2 * d * page))
        self.table = torch.cat([self.table, torch.full((len(qs), columns), 1 << 30, dtype=torch.int32)], 1)
        self.dev[0] = self.table.cuda()

    def call(self, q, groups=None, **kw):
        groups = groups or (ints(self.group_cu), ints(self.prefixes))
        return nv.nvfp4_attn_paged_shared(q, *self.args(), *groups, max(self.qs + [1]), **kw)


def check(p, q, gate=None, scale=None, error=0, **kw):
    y = p.call(q, gate=gate, scale=scale, **kw)
    assert nv.nvfp4_device_error() == error
    ref, size = attn64(p, q.cpu(), p.d ** -0.5 if scale is None else scale, None if gate is None else gate.cpu())
    close_bf16(y, ref, 2.0 ** -8 * size)
    return y


def queries(p, g, size=1.5):
    return (randn(p.g, sum(p.qs), g * p.hkv, p.d) * size).bfloat16().cuda()


CASES = [
    # one group: few rows (kernel for few rows in both passes), a copy a quarter or half, several blocks
    ([1, 1], [300, 270], [0, 2], [256], 1, 1, 128, 16), ([1] * 4, [200, 140, 333, 129], [0, 4], [128], 4, 2, 64, 16),
    ([1] * 7, [700 + 9 * i for i in range(7)], [0, 7], [640], 4, 2, 128, 64), ([1] * 13, [600] * 13, [0, 13], [512], 4, 1, 96, 32),
    ([1] * 40, [1500 + i for i in range(40)], [0, 40], [1408], 5, 2, 128, 64), ([1] * 9, [2000] * 9, [0, 9], [1984], 6, 4, 256, 64),
    ([2] * 20, [900 + 3 * i for i in range(20)], [0, 20], [800], 8, 1, 256, 16),
    # prompts of their own behind the prefix
    ([30, 70, 1], [700, 800, 650], [0, 3], [640], 3, 2, 128, 64), ([130, 257], [900, 1000], [0, 2], [640], 4, 1, 128, 128),
    ([100, 33], [640, 700], [0, 2], [512], 6, 1, 256, 256), ([50] * 5, [450] * 5, [0, 5], [384], 2, 2, 80, 32),
    # several blocks of rows a sequence
    ([5, 3, 7], [700, 702, 650], [0, 3], [640], 9, 1, 128, 16), ([3] * 6, [500 + 11 * i for i in range(6)], [0, 6], [384], 8, 2, 256, 64),
    ([7, 1, 4], [400, 420, 390], [0, 3], [256], 9, 1, 256, 32), ([20, 2], [340, 350], [0, 2], [256], 3, 2, 96, 64),
    # several groups, sequences of no group before, between and behind, empty groups, sequences that bring nothing
    ([1] * 8, [300, 700, 720, 50, 900, 901, 910, 40], [1, 3, 3, 7], [640, 512, 384], 4, 2, 128, 64),
    ([3, 0, 2, 5, 1, 0, 4, 8, 1], [400, 380, 500, 260, 300, 0, 700, 650, 90], [0, 3, 5, 8], [256, 256, 640], 6, 1, 256, 32),
    ([1] * 30, [256 + 128 * (i // 6) + i for i in range(30)], [0, 6, 12, 18, 24, 30], [256, 384, 512, 640, 768], 4, 1, 128, 16),
    # prefixes that cannot be shared whole: beyond what a sequence holds, no whole tile, one sequence, nothing held, no place
    ([1, 1, 1], [1000, 400, 700], [0, 3], [960], 4, 2, 128, 64), ([2, 2], [200, 220], [0, 2], [96], 4, 2, 128, 16),
    ([1, 1], [600, 650], [0, 1, 2], [512, 640], 4, 1, 128, 64), ([1, 1, 1], [600, 0, 640], [0, 3], [512], 4, 1, 128, 64),
    ([4, 4, 4], [600, 2, 640], [0, 3], [512], 2, 1, 128, 64), ([1, 1], [128, 257], [0, 2], [128], 4, 1, 64, 16),
    ([1, 1], [129, 257], [0, 2], [128], 4, 1, 64, 16), ([5, 5], [133, 140], [0, 2], [128], 1, 3, 16, 128),
]


@pytest.mark.parametrize("qs,kvs,groups,prefixes,g,hkv,d,page", CASES)
def test_shared_prefixes(qs, kvs, groups, prefixes, g, hkv, d, page):
    p = Shared(sum(kvs) + d, qs, kvs, groups, prefixes, hkv, d, page)
    q = queries(p, g)
    gate = randn(p.g, *q.shape).bfloat16().cuda()
    check(p, q)
    check(p, q, gate=gate, max_own_len=300, max_group_tokens=sum(qs))
    check(p, q, gate=gate, max_kv_len=max(kvs))  # not worth it


def test_long_prefix_and_long_own_parts():
    """Blocks of many parts in both passes."""
    p = Shared(1, [1] * 6, [20000, 20100, 27000, 20480, 24000, 20481], [0, 6], [19968], 1, 128, 64)
    check(p, queries(p, 8))
    p = Shared(2, [2, 1], [30000, 30500], [0, 2], [29000], 2, 128, 64)  # few rows
    check(p, queries(p, 4), max_own_len=100)  # a bound that does not hold chooses kernels, no more
    p = Shared(3, [1] * 5, [9000, 9001, 9002, 9003, 9004], [0, 5], [8960], 2, 256, 64)
    check(p, queries(p, 6))


@pytest.mark.parametrize("b,own,hkv,d,page", [(48, 1000, 4, 64, 32), (64, 2600, 8, 16, 256)])
def test_chunks_of_many_steps(b, own, hkv, d, page):
    """So many tokens that chunks get longer than the shortest, and than the 32 steps whose pages are looked up at once."""
    p = Shared(b, [1] * b, [256 + own + 13 * i for i in range(b)], [0, b], [256], hkv, d, page)
    check(p, queries(p, 2))


@pytest.mark.parametrize("groups,each,hkv,d,own", [(40, 2, 8, 128, 40), (25, 3, 8, 256, 300), (3, 2, 1, 128, 20), (7, 4, 4, 256, 900),
                                                   (2, 16, 8, 64, 1500)])
def test_blocks_of_a_part_of_the_grid_or_of_more(groups, each, hkv, d, own):
    """Blocks that have CTAs of their own, and more blocks than CTAs; chunks that are all taken at once, or in turns."""
    b = groups * each
    prefixes = [256 + 128 * (i % 5) for i in range(groups)]
    kvs = [prefixes[i // each] + 1 + own * (i % 7 + 1) // 7 for i in range(b)]
    p = Shared(b + d, [1 + i % 2 for i in range(b)], kvs, list(range(0, b + 1, each)), prefixes, hkv, d, 64)
    check(p, queries(p, 3))


def test_sequences_that_claim_the_same_rows():
    """A cu_q that cannot be used, in which 4000 sequences claim rows 0 to 3: more parts than there is room for."""
    b = 8000
    p = Shared(1, [4] * 4, [200] * 4, [0, 4], [128], 1, 256, 64)
    q = queries(p, 8)
    table = p.dev[0][:1].expand(b, -1).contiguous()
    cu, kv = ints([0, 4] * (b // 2) + [0]), ints([200] * b)
    y = nv.nvfp4_attn_paged_shared(q, *p.args()[:4], table, cu, kv, ints([0, 4]), ints([128]), 4)
    assert nv.nvfp4_device_error() == 256
    assert torch.isfinite(y[:4]).all()
    check(p, q)


@pytest.mark.parametrize("qs,kvs,d", [([1] * 5, [520, 540, 513, 600, 700], 128), ([40] * 3, [560, 700, 600], 256)])
def test_group_tokens_beyond_the_bound_share_nothing(qs, kvs, d):
    p = Shared(7, qs, kvs, [0, len(qs)], [512], 1, d, 64)
    check(p, queries(p, 4), max_group_tokens=2)


def test_no_groups_is_attention_as_it_is():
    p = Shared(8, [1, 3], [300, 500], [0], [], 2, 128, 32)
    q = queries(p, 4)
    assert torch.equal(check(p, q), nv.nvfp4_attn_paged(q, *p.args(), 3))


@pytest.mark.parametrize("groups,prefixes", [([0, 3, 2], [256, 256]), ([-1, 2], [256]), ([0, 9], [256]), ([2, 1], [256])])
def test_groups_that_cannot_be_used_share_nothing(groups, prefixes):
    p = Shared(9, [1] * 8, [300 + 10 * i for i in range(8)], [0, 4, 8], [256, 256], 1, 128, 64)
    p.group_cu, p.prefixes = groups, prefixes
    check(p, queries(p, 4), error=256)


@pytest.mark.parametrize("length", [-1, 420_001, 1 << 30])
def test_prefix_lengths_that_cannot_be_used_share_nothing(length):
    p = Shared(9, [1] * 4, [300, 310, 320, 330], [0, 4], [256], 1, 128, 64)
    p.prefixes = [length]
    check(p, queries(p, 4), error=256, max_kv_len=420_000)


def test_bad_paging_data():
    p = Shared(10, [1] * 4, [300, 310, 320, 330], [0, 4], [256], 1, 128, 64)
    q = queries(p, 4)
    check(p, q)
    # a sequence that cannot be used is passed over, and its group shares nothing
    for cu in ([0, 1, 5, 3, 4], [0, 1, 1, 4, 5]):
        out = torch.full_like(q, 7.0)
        nv.nvfp4_attn_paged_shared(q, *p.args()[:5], ints(cu), p.dev[2], ints([0, 4]), ints([256]), 2, out=out)
        assert nv.nvfp4_device_error() == 256
        want = torch.full_like(q, 7.0)
        nv.nvfp4_attn_paged(q, *p.args()[:5], ints(cu), p.dev[2], 2, out=want)
        assert nv.nvfp4_device_error() == 256
        assert torch.equal(out == 7.0, want == 7.0)
        far = (out.double() - want.double()).abs() - 2.0 ** -7 * want.double().abs()  # either is off by half of that
        assert float(far.max()) <= 2.0 ** -7 * float((p.v.double() * p.vs[:, :, None, None].double()).abs().max())
    # one that holds an unusable number of tokens holds nothing; the others share on
    y = nv.nvfp4_attn_paged_shared(q, *p.args()[:6], ints([300, -5, 320, 330]), ints([0, 4]), ints([256]), 1)
    assert nv.nvfp4_device_error() == 256
    p.kvs[1] = 0
    ref, size = attn64(p, q.cpu(), p.d ** -0.5)
    close_bf16(y, ref, 2.0 ** -8 * size)
    assert not y[1].any()
    # pages that are none read as zeros
    t = p.dev[0].clone()
    t[:, 1] = p.pages
    y = nv.nvfp4_attn_paged_shared(q, *p.args()[:4], t, *p.dev[1:], ints([0, 4]), ints([256]), 1)
    assert nv.nvfp4_device_error() == 256 and torch.isfinite(y).all()


@pytest.mark.parametrize("n,d,g", [(1, 128, 4), (1, 256, 6), (1, 128, 30), (60, 128, 4), (60, 256, 2)])
def test_what_nobody_sees_may_be_anything(n, d, g):
    """NaN in slots behind the last token, in unused pages and their scales, and in rows of the padded batch."""
    p = Shared(n + d, [n] * 4, [n + 256 + 5, n + 256 + 70, 0, n + 256], [0, 4], [256], 1, d, 64)
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
    q = queries(p, g)
    gate = randn(p.g, *q.shape).bfloat16().cuda()
    y = check(p, q, gate=gate)
    q[2 * n:3 * n] = math.nan  # the sequence that holds nothing
    gate[2 * n:3 * n] = math.nan
    assert torch.equal(p.call(q, gate=gate), y)


@pytest.mark.parametrize("n,d,g", [(1, 128, 2), (1, 128, 9), (1, 128, 40), (2, 256, 12), (50, 128, 4)])
def test_what_is_not_finite_reaches_the_rows_that_see_it(n, d, g):
    p = Shared(n * d, [n] * 4, [n + 384 + i for i in range(4)], [0, 4], [384], 1, d, 32)
    q = queries(p, g)
    y = check(p, q)
    bad = q.clone()
    bad[n, 1, 3] = math.inf  # one row
    z = p.call(bad)
    hit = torch.zeros(z.shape[:2], dtype=torch.bool, device="cuda")
    hit[n, 1] = True
    assert torch.isnan(z[hit]).all() and torch.equal(z[~hit], y[~hit])
    page, slot = int(p.table[0, 5]), 7  # of the prefix: all rows
    v = p.v.view(torch.uint8)
    old = v[page, 0, slot, 7].item()
    v[page, 0, slot, 7] = 0x7F
    z = p.call(q)
    assert torch.isnan(z[:, :, 7]).all() and torch.equal(z[..., 8:], y[..., 8:]) and torch.equal(z[..., :7], y[..., :7])
    v[page, 0, slot, 7] = old
    own = int(p.table[2, 12])  # the first page behind the prefix, of the third sequence
    v[own, 0, 0, 9] = 0xFF
    z = p.call(q)
    assert torch.isnan(z[2 * n:3 * n, :, 9]).all()
    z[2 * n:3 * n, :, 9] = y[2 * n:3 * n, :, 9]
    assert torch.equal(z, y)


@pytest.mark.parametrize("g", [4, 40])
def test_one_side_far_above_the_other(g):
    """All of a row's weight in the prefix, or in its own tokens, and scales of any size."""
    p = Shared(5, [1] * 4, [300, 310, 320, 330], [0, 4], [256], 1, 128, 16)
    q = queries(p, g, 1.0)
    for factor in (2.0 ** 7, 2.0 ** -7):
        p.ks[p.table[0, :16].long().cuda()] *= factor
        check(p, q)
    p.vs.copy_((2.0 ** torch.randint(-90, 90, p.vs.shape, generator=p.g).float()).cuda())
    check(p, q)


@pytest.mark.parametrize("layout", ["slice", "heads_first", "odd"])
@pytest.mark.parametrize("n,kvs", [(1, [300, 290]), (45, [400, 390])])
def test_row_layouts_and_scale(layout, n, kvs):
    p = Shared(n, [n, n], kvs, [0, 2], [256], 2, 128, 16, layout="tokens_first")
    q, gate = rows(p.g, 2 * n, 6, 128, layout), rows(p.g, 2 * n, 6, 128, layout)
    check(p, q, gate=gate, scale=0.2)


@pytest.mark.parametrize("qs,kvs,prefix,g,d", [([1] * 12, [5000 + 31 * i for i in range(12)], 4992, 4, 128),
                                               ([1] * 3, [9000, 8000, 8300], 7936, 4, 128), ([90, 40], [2200, 2300], 2048, 4, 256)])
def test_same_bits_every_time_on_other_streams_and_workspaces(qs, kvs, prefix, g, d):
    p = Shared(sum(kvs), qs, kvs, [0, len(qs)], [prefix], 2, d, 64)
    q = queries(p, g)
    y = check(p, q)
    size = nv.nvfp4_attn_shared_workspace_size(sum(qs), 2 * g, d, len(p.qs))
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN, whatever it is read as
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        with torch.cuda.stream(s):
            a = p.call(q)
            b = p.call(q, workspace=ws)
        c = p.call(q)
        torch.cuda.synchronize()
        assert torch.equal(a, y) and torch.equal(b, y) and torch.equal(c, y)
    with pytest.raises(nv.Nvfp4Error, match="needed"):
        p.call(q, workspace=ws[:-256])


def test_rows_behind_the_last_sequence_stay():
    p = Shared(3, [1, 1, 1], [300, 310, 320], [0, 3], [256], 1, 128, 64)
    q = randn(p.g, 6, 4, 128).bfloat16().cuda()
    out = torch.full_like(q, 7.0)
    y = p.call(q, out=out, max_group_tokens=3)  # (else the bound is 6, and chooses another kernel)
    assert y.data_ptr() == out.data_ptr() and (out[3:] == 7.0).all()
    assert torch.equal(out[:3], p.call(q[:3].contiguous()))


def test_a_captured_step_replays_as_sequences_grow():
    p = Shared(21, [1] * 6, [400] * 6, [0, 6], [256], 2, 128, 16)
    kv = ints([300 + i for i in range(6)])
    p.dev[2] = kv
    q = queries(p, 4)
    groups = ints(p.group_cu), ints(p.prefixes)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        p.call(q, groups)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y = p.call(q, groups)
    for _ in range(5):
        q.copy_(queries(p, 4))
        kv.add_(13)
        graph.replay()
        torch.cuda.synchronize()
        p.kvs = kv.tolist()
        ref, size = attn64(p, q.cpu(), 128 ** -0.5)
        close_bf16(y, ref, 2.0 ** -8 * size)


def test_empty_calls_do_nothing():
    p = Shared(1, [0], [5], [0, 1], [0], 1, 32, 16)
    q = torch.empty((0, 2, 32), dtype=torch.bfloat16, device="cuda")
    assert p.call(q).shape == (0, 2, 32)


@pytest.mark.parametrize("qs,kvs,prefix,g,d", [([1] * 41, [300 + 9 * i for i in range(41)], 256, 5, 256),
                                               ([1] * 5, [130, 140, 150, 160, 170], 128, 4, 128), ([20, 9], [160, 150], 128, 4, 256)])
@pytest.mark.parametrize("byte", [0x00, 0x7F, 0x80, 0xFF])
def test_few_units_and_any_workspace(qs, kvs, prefix, g, d, byte):
    p = Shared(sum(kvs) + d, qs, kvs, [0, len(qs)], [prefix], 1, d, 32)
    size = nv.nvfp4_attn_shared_workspace_size(sum(qs), g, d, len(p.qs))
    check(p, queries(p, g), workspace=torch.full((size,), byte, dtype=torch.uint8, device="cuda"))
