"""Refusals of the block tables', the shared prefixes' and the verification's entry points: host only, no GPU."""
from __future__ import annotations

import pytest
import torch

import nvfp4_weight_quantized_gemv_gb300 as nv
from test_attention_abi import BAD_BATCH, BAD_CACHE, batch, built, cache, rows  # noqa: F401

A = 4096  # an address that nothing reads


def pages(table=A, stride=8, width=8, page=16, free=A, ring=64, span=A, span_out=A, held=A, held_out=A, kept=None):
    return nv.nvfp4_kv_pages(table, stride, width, page, free, ring, span, span_out, held, held_out, kept)


def tables(p, b=4, kv=A, q=A, tokens=8, cu=A, lens=A, pos=A, slots=A):
    return nv.lib().nvfp4_kv_tables(p, b, kv, q, tokens, cu, lens, pos, slots, None)


@pytest.mark.parametrize("p,status", [
    (dict(table=None), 1), (dict(width=0), 1), (dict(stride=7), 1), (dict(stride=-1), 1), (dict(page=8), 1), (dict(page=48), 1),
    (dict(page=512), 1), (dict(free=None), 1), (dict(ring=0), 1), (dict(ring=(1 << 30) + 1), 1), (dict(span=None), 1),
    (dict(span_out=None), 1), (dict(held=None), 1), (dict(held_out=None), 1), (dict(width=(1 << 26) + 1, stride=1 << 28), 1),
    (dict(table=A + 2), 2), (dict(span=A + 4), 2), (dict(span_out=A + 4), 2), (dict(kept=A + 1), 2), (dict(held=A + 1), 2)])
def test_bad_pages(p, status):
    assert tables(pages(**p)) == status
    assert nv.nvfp4_last_error()


@pytest.mark.parametrize("a,status", [
    (dict(b=-1), 1), (dict(b=8193), 1), (dict(kv=None), 1), (dict(q=None), 1), (dict(tokens=-1), 1),
    (dict(tokens=(1 << 30) + 1), 1), (dict(cu=None), 1), (dict(lens=None), 1), (dict(pos=None), 1), (dict(slots=None), 1),
    (dict(slots=A + 4), 2), (dict(cu=A + 1), 2), (dict(pos=A + 2), 2)])
def test_bad_table_arguments(a, status):
    assert tables(pages(), **a) == status
    assert tables(None) == 1


def draft_rows(target=A, draft=A, ts=100, ds=100, ids=A, tokens=4, vocab=100):
    return nv.nvfp4_draft_rows(target, draft, ts, ds, ids, tokens, vocab)


def verify(r, cu=A, kv=A, u=A, pick=A, b=2, out=A, acc=A, nxt=A, lens=A):
    return nv.lib().nvfp4_verify_drafts(r, cu, kv, u, pick, b, out, acc, nxt, lens, None)


@pytest.mark.parametrize("r,status", [
    (dict(target=None), 1), (dict(ts=-1), 1), (dict(ds=-4), 1), (dict(ids=None), 1), (dict(tokens=-1), 1),
    (dict(tokens=(1 << 30) + 1), 1), (dict(vocab=0), 1), (dict(vocab=(1 << 30) + 1), 1), (dict(target=A + 2), 2),
    (dict(draft=A + 1), 2), (dict(ids=A + 2), 2)])
def test_bad_draft_rows(r, status):
    assert verify(draft_rows(**r)) == status
    assert nv.nvfp4_last_error()


@pytest.mark.parametrize("a,status", [
    (dict(cu=None), 1), (dict(u=None), 1), (dict(pick=None), 1), (dict(b=-1), 1), (dict(b=65536), 1), (dict(out=None), 1),
    (dict(acc=None), 1), (dict(nxt=None), 1), (dict(lens=None), 1), (dict(u=A + 2), 2), (dict(lens=A + 3), 2)])
def test_bad_verification_arguments(a, status):
    assert verify(draft_rows(), **a) == status
    assert verify(None) == 1
    assert verify(draft_rows(), b=0, cu=None, u=None) == nv.NVFP4_OK


def prefix(cu=A, lens=A, groups=1, most=4, own=16):
    return nv.nvfp4_kv_prefix(cu, lens, groups, most, own)


def shared(q=rows(), c=None, n=None, p=None, scale=1.0, gate=None, y=A, ws=A, nb=1 << 40):
    return nv.lib().nvfp4_attn_paged_shared(q, c or cache(), n or batch(), p or prefix(), scale, gate, y, ws, nb, None)


@pytest.mark.parametrize("p,status", [(dict(cu=None), 1), (dict(lens=None), 1), (dict(groups=-1), 1), (dict(groups=3), 1),
                                      (dict(most=0), 1), (dict(own=-1), 1), (dict(cu=A + 2), 2), (dict(lens=A + 1), 2)])
def test_bad_prefixes(p, status):
    assert shared(p=prefix(**p)) == status
    assert nv.nvfp4_last_error()


def test_shared_attention_refuses_what_attention_refuses():
    for c, status in BAD_CACHE:
        assert shared(c=cache(**c)) == status
    for n, status in BAD_BATCH:
        assert shared(n=batch(**n)) == status
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert shared(scale=scale) == 1
    assert shared(q=None) == 1 and shared(y=None) == 1 and shared(y=A + 8) == 2 and shared(q=rows(heads=3)) == 1
    assert shared(gate=rows(heads=2)) == 1 and shared(ws=None) == 1 and shared(ws=A + 16) == 1
    assert nv.lib().nvfp4_attn_paged_shared(rows(), cache(), batch(), None, 1.0, None, A, A, 1 << 40, None) == 1
    assert shared(n=batch(b=0), q=None, y=None, ws=None, p=prefix(groups=0)) == nv.NVFP4_OK


def test_shared_workspace_size():
    size = nv.nvfp4_attn_shared_workspace_size
    assert size(0, 8, 64, 0) >= nv.nvfp4_attn_workspace_size()
    assert size(1000, 8, 128, 10) >= size(0, 8, 128, 0) + 1000 * 8 * (4 * 128 + 8) + 640
    assert size(1 << 20, 64, 256, 65535) > 1 << 36  # in 64 bits
    for bad in ((-1, 8, 64, 1), (1, 0, 64, 1), (1, 8, 72, 1), (1, 8, 64, 65536), (1, 8, 64, -1)):
        with pytest.raises(nv.Nvfp4Error):
            size(*bad)


def test_python_checks():
    i = torch.zeros(2, 4, dtype=torch.int32)
    f = torch.zeros(3, 8)
    with pytest.raises(TypeError, match="block_table"):
        nv.nvfp4_kv_tables(i, i[0, :2], i[0], torch.zeros(2, dtype=torch.int64), i[0, :2], i[0, :2], 16, 4)
    with pytest.raises(TypeError, match="target"):
        nv.nvfp4_verify_drafts(f, i[0, :3], i[0, :2], f[:, 0], f[0, :1])
    with pytest.raises(TypeError, match="CUDA bfloat16"):
        x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
        nv.nvfp4_attn_paged_shared(x, x, x, x, x, i, i, i, i, i, 1)
