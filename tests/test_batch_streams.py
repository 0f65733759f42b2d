"""Streams and devices of the block tables, the shared prefixes and the verification, and caches beyond 4 GB."""
from __future__ import annotations

import pytest
import torch

import nvfp4_weight_quantized_gemv_gb300 as nv
from test_attention_ops import attn64, built, close_bf16, randn  # noqa: F401
from test_shared_prefix import Shared, ints, queries
from test_streams import Elsewhere, freed

pytestmark = pytest.mark.gpu


def on_its_stream(call, like):
    """call(stream): its first output is of memory of `stream`, and right there."""
    side = torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        here, there = freed(like, torch.cuda.current_stream()), freed(like, side)
        got = call(handle)
        assert got[0].untyped_storage().data_ptr() == there != here
        with torch.cuda.stream(side):
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        del got
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


def bytes_like(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def test_outputs_are_allocated_on_their_stream():
    t = 1 << 20
    table, held, ring = torch.zeros(2, 1 << 16, dtype=torch.int32).cuda(), ints([0, 0]), torch.arange(1 << 17).int().cuda()
    span = torch.tensor([0, 1 << 17]).cuda()
    on_its_stream(lambda s: nv.nvfp4_kv_tables(table, held, ring, span, ints([0, 0]), ints([t // 2, 5]), 16, t, stream=s),
                  bytes_like(12 * t + 80))
    rows = 1 << 18
    p = torch.rand(2, 64).cuda().repeat(rows // 2, 1)
    ids, u = torch.zeros(rows, dtype=torch.int32).cuda(), torch.rand(rows).cuda()
    cu, pick = torch.arange(0, rows + 1, 8).int().cuda(), torch.rand(rows // 8).cuda()
    on_its_stream(lambda s: [nv.nvfp4_verify_drafts(p, ids, cu, u, pick, stream=s)[0]], bytes_like(4 * rows + 8 * (rows // 8)))
    p = Shared(2, [1] * 8, [300 + i for i in range(8)], [0, 8], [256], 1, 64, 64)
    x = queries(p, 8).repeat(4096, 1, 1)  # rows behind the last sequence, for a large output
    out = lambda s: [nv.nvfp4_attn_paged_shared(x, *p.args(), ints([0, 8]), ints([256]), 1, stream=s)[:8]]  # noqa: E731
    on_its_stream(out, torch.empty_like(x))


def test_calls_on_two_streams_at_once():
    p = Shared(3, [1] * 20, [400 + i for i in range(20)], [0, 20], [256], 2, 128, 64)
    r = Shared(4, [2] * 9, [700 + i for i in range(9)], [0, 9], [640], 2, 256, 32)
    work = [(p, queries(p, 4)), (r, queries(r, 6))]
    want = [c.call(q) for c, q in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for i, (c, q) in enumerate(work):
            with torch.cuda.stream(streams[i]):
                got[i].append(c.call(q))
    torch.cuda.synchronize()
    for a, all_ in zip(want, got):
        assert all(torch.equal(a, b) for b in all_)
    assert nv.nvfp4_device_error() == 0


def test_tensors_of_another_device_are_refused():
    p = Shared(3, [1, 1], [300, 310], [0, 2], [256], 1, 128, 64)
    q = queries(p, 2)
    ws = torch.empty(nv.nvfp4_attn_shared_workspace_size(2, 2, 128, len(p.qs)), dtype=torch.uint8, device="cuda")
    span, t = torch.tensor([0, 4]).cuda(), torch.rand(3, 50).cuda()

    def shared(q, kc, vc, ks, vs, table, cu, lens, group, prefix, gate, out, ws):
        nv.nvfp4_attn_paged_shared(q, kc, vc, ks, vs, table, cu, lens, group, prefix, 1, gate=gate, out=out, workspace=ws)

    def tables(table, held, ring, span, kv, q_lens, kept, held_out, span_out):
        nv.nvfp4_kv_tables(table, held, ring, span, kv, q_lens, 16, 8, kept=kept, held_out=held_out, span_out=span_out)

    def verify(target, ids, cu, u, pick, draft, lens):
        nv.nvfp4_verify_drafts(target, ids, cu, u, pick, draft=draft, kv_lens=lens)

    def other(x):
        return Elsewhere._make_wrapper_subclass(Elsewhere, x.size(), x.stride(), dtype=x.dtype, device=torch.device("cuda:1"))

    two = lambda: ints([0, 0])  # noqa: E731
    for call, args in ((shared, [q, *p.args(), ints([0, 2]), ints([256]), q, torch.empty_like(q), ws]),
                       (tables, [torch.zeros(2, 4, dtype=torch.int32).cuda(), two(), ints([1, 2, 3, 4]), span, two(), two(), two(),
                                 two(), span.clone()]),
                       (verify, [t, ints([1, 2, 3]), ints([0, 2, 3]), t[:, 0].contiguous(), t[0, :2].contiguous(), t, two()])):
        call(*args)
        for i in range(len(args)):
            with pytest.raises(ValueError, match="is on cuda:1, the current device is cuda:0"):
                call(*args[:i], other(args[i]), *args[i + 1:])
    assert nv.nvfp4_device_error() == 0


def test_arguments_of_other_shapes_and_types_are_refused():
    p = Shared(3, [1, 1], [300, 310], [0, 2], [256], 1, 128, 64)
    q = queries(p, 2)
    for group, prefix in ((ints([0, 2, 2]), ints([256])), (ints([0, 2]).long(), ints([256])), (ints([0, 2]), ints([256]).float()),
                          (ints([[0, 2]]), ints([256])), (ints([0, 1, 2, 2, 2, 2]), ints([256, 0, 0, 0, 0]))):
        with pytest.raises((TypeError, ValueError, nv.Nvfp4Error)):
            nv.nvfp4_attn_paged_shared(q, *p.args(), group, prefix, 1)
    table, two, span = torch.zeros(2, 4, dtype=torch.int32).cuda(), ints([0, 0]), torch.tensor([0, 3]).cuda()
    good = [table, two, ints([1, 2, 3]), span, two, two, 16, 5]
    nv.nvfp4_kv_tables(*good)
    for i, bad in ((0, table.t()), (0, table.long()), (0, table[0]), (1, ints([0])), (1, two.long()), (2, ints([[1, 2]])),
                   (3, span.int()), (3, span[:1]), (4, ints([0, 0, 0])), (5, ints([0])), (6, 24), (7, -1), (2, ints([]))):
        with pytest.raises((TypeError, ValueError, nv.Nvfp4Error)):
            nv.nvfp4_kv_tables(*good[:i], bad, *good[i + 1:])
    with pytest.raises((ValueError, nv.Nvfp4Error)):
        nv.nvfp4_kv_tables(table[:1].expand(2, 4), *good[1:])  # two sequences, one row
    t = torch.rand(3, 50).cuda()
    good = [t, ints([1, 2, 3]), ints([0, 3]), t[:, 0].contiguous(), t[0, :1].contiguous(), t]
    call = lambda a: nv.nvfp4_verify_drafts(*a[:5], draft=a[5])  # noqa: E731
    call(good)
    for i, bad in ((0, t.half()), (0, t.t()), (0, t[0]), (1, ints([1, 2])), (1, ints([1, 2, 3]).long()), (2, ints([0])),
                   (3, t[:2, 0].contiguous()), (4, t[0, :2].contiguous()), (5, t[:2]), (5, t.double()), (5, t[:, :49])):
        with pytest.raises((TypeError, ValueError, nv.Nvfp4Error)):
            call([*good[:i], bad, *good[i + 1:]])
    assert nv.nvfp4_device_error() == 0


def test_pages_beyond_4_gb():
    """Pages 1 GB apart: the offsets of the later ones do not fit 32 bits."""
    p = Shared(6, [1, 1, 1], [140, 150, 161], [0, 3], [128], 1, 64, 64, spare=0)
    step, n = 1 << 30, p.pages
    big = torch.empty(step * (n - 1) + 2 * 64 * 64, dtype=torch.uint8, device="cuda")
    k, v = (torch.as_strided(big, (n, 1, 64, 64), (step, 64 * 64, 64, 1), at) for at in (0, 64 * 64))
    k.copy_(p.k.view(torch.uint8)), v.copy_(p.v.view(torch.uint8))
    q = queries(p, 4)
    y = nv.nvfp4_attn_paged_shared(q, k, v, p.ks, p.vs, *p.dev, ints([0, 3]), ints([128]), 1)
    assert torch.equal(y, p.call(q))
    ref, size = attn64(p, q.cpu(), 64 ** -0.5)
    close_bf16(y, ref, 2.0 ** -8 * size)
    assert nv.nvfp4_device_error() == 0
