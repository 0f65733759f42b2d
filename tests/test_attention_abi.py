"""Refusals of the attention operators' entry points: host only, no GPU."""
from __future__ import annotations

import ctypes

import pytest
import torch

import nvfp4_weight_quantized_gemv_gb300 as nv


@pytest.fixture(scope="module", autouse=True)
def built():
    nv.build()


def rows(p=4096, ts=512, hs=64, heads=4):
    return nv.nvfp4_head_rows(p, ts, hs, heads)


def how(qw=None, kw=None, eps=1e-6, cs=4096, positions=64, rot=64, inter=0):
    return nv.nvfp4_norm_rope(qw, kw, eps, cs, positions, rot, inter)


def cache(k=4096, v=4096, ks=4096, vs=4096, ps=4096, hs=1024, ts=64, pages=8, heads=2, page=16, d=64):
    return nv.nvfp4_kv_cache(k, v, ks, vs, ps, hs, ts, pages, heads, page, d)


def batch(table=4096, cu=4096, kv=4096, b=2, stride=4, tokens=2, max_q=1, max_kv=64):
    return nv.nvfp4_kv_batch(table, cu, kv, b, stride, tokens, max_q, max_kv)


BAD_CACHE = [(dict(k=None), 1), (dict(vs=None), 1), (dict(page=24), 1), (dict(page=512), 1), (dict(page=8), 1),
             (dict(d=72), 1), (dict(d=272), 1), (dict(d=0), 1), (dict(pages=0), 1), (dict(heads=0), 1),
             (dict(ts=48), 1), (dict(ps=-16), 1), (dict(k=4104), 2), (dict(ts=72), 2), (dict(ps=4104), 2),
             (dict(ks=4097), 2)]
BAD_BATCH = [(dict(b=-1), 1), (dict(tokens=-1), 1), (dict(table=None), 1), (dict(cu=None), 1), (dict(kv=None), 1),
             (dict(max_q=0), 1), (dict(max_kv=65), 1), (dict(max_kv=-1), 1), (dict(stride=0), 1), (dict(b=70000), 1)]


@pytest.mark.parametrize("c,status", BAD_CACHE)
def test_bad_caches(c, status):
    L = nv.lib()
    kv = rows(heads=2)
    assert L.nvfp4_kv_append(None, kv, kv, how(), cache(**c), batch(), None, None) == status
    assert L.nvfp4_attn_paged(rows(), cache(**c), batch(), 1.0, None, 4096, None, 0, None) == status
    assert nv.nvfp4_last_error()


@pytest.mark.parametrize("n,status", BAD_BATCH)
def test_bad_batches(n, status):
    L = nv.lib()
    kv = rows(heads=2)
    assert L.nvfp4_kv_append(None, kv, kv, how(), cache(), batch(**n), None, None) == status
    assert L.nvfp4_attn_paged(rows(), cache(), batch(**n), 1.0, None, 4096, None, 0, None) == status


@pytest.mark.parametrize("h,status", [(dict(rot=63), 1), (dict(rot=66), 1), (dict(rot=-2), 1), (dict(cs=None), 1),
                                      (dict(positions=0), 1), (dict(inter=2), 1), (dict(qw=4096, eps=-1.0), 1),
                                      (dict(kw=4096, eps=float("nan")), 1), (dict(cs=4098), 2), (dict(qw=4097), 2)])
def test_bad_norm_and_rotation(h, status):
    L = nv.lib()
    kv = rows(heads=2)
    assert L.nvfp4_qk_norm_rope(rows(), None, 4096, how(**h), 2, 64, 4096, None, None) == status
    assert L.nvfp4_kv_append(None, kv, kv, how(**h), cache(), batch(), None, None) == status


@pytest.mark.parametrize("r,status", [(dict(p=None), 1), (dict(heads=0), 1), (dict(ts=-1), 1), (dict(hs=-64), 1),
                                      (dict(p=4097), 2), (dict(heads=3), 1)])
def test_bad_rows(r, status):
    L = nv.lib()
    kv = rows(heads=2)
    bad = dict(dict(heads=2), **r)
    assert L.nvfp4_kv_append(None, rows(**bad), kv, how(), cache(), batch(), None, None) == status
    assert L.nvfp4_kv_append(None, kv, rows(**bad), how(), cache(), batch(), None, None) == status
    assert L.nvfp4_attn_paged(rows(**bad), cache(), batch(), 1.0, None, 4096, None, 0, None) == status
    assert L.nvfp4_attn_paged(rows(), cache(), batch(), 1.0, rows(**bad), 4096, None, 0, None) == status


def test_other_refusals():
    L = nv.lib()
    kv = rows(heads=2)
    norm = lambda q, k, pos, tokens, d, qo, ko: L.nvfp4_qk_norm_rope(q, k, pos, how(), tokens, d, qo, ko, None)  # noqa: E731
    assert norm(None, None, 4096, 2, 64, 4096, None) == nv.NVFP4_ERR_INVALID_ARG
    assert norm(rows(), None, None, 2, 64, 4096, None) == nv.NVFP4_ERR_INVALID_ARG
    assert norm(rows(), rows(), 4096, 2, 64, 4096, None) == nv.NVFP4_ERR_INVALID_ARG
    assert norm(rows(), None, 4096, 2, 72, 4096, None) == nv.NVFP4_ERR_INVALID_ARG
    assert norm(rows(), None, 4096, -1, 64, 4096, None) == nv.NVFP4_ERR_INVALID_ARG
    assert norm(rows(), None, 4096, 2, 64, 4100, None) == nv.NVFP4_ERR_MISALIGNED
    assert L.nvfp4_qk_norm_rope(rows(), None, 4096, None, 2, 64, 4096, None, None) == nv.NVFP4_ERR_INVALID_ARG
    append = lambda q, n, h, qo: L.nvfp4_kv_append(q, kv, kv, h, cache(), n, qo, None)  # noqa: E731
    assert append(rows(), batch(), how(), None) == nv.NVFP4_ERR_INVALID_ARG
    assert append(rows(), batch(), how(), 4104) == nv.NVFP4_ERR_MISALIGNED
    assert append(None, batch(), how(positions=63), None) == nv.NVFP4_ERR_INVALID_ARG
    assert L.nvfp4_kv_append(None, None, kv, how(), cache(), batch(), None, None) == nv.NVFP4_ERR_INVALID_ARG
    attn = lambda q=rows(), scale=1.0, y=4096, ws=None, nb=0: L.nvfp4_attn_paged(  # noqa: E731
        q, cache(), batch(), scale, None, y, ws, nb, None)
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert attn(scale=bad) == nv.NVFP4_ERR_INVALID_ARG
    assert attn(q=None) == nv.NVFP4_ERR_INVALID_ARG and attn(y=None) == nv.NVFP4_ERR_INVALID_ARG
    assert attn(y=4104) == nv.NVFP4_ERR_MISALIGNED and attn(ws=4104, nb=1 << 30) == nv.NVFP4_ERR_INVALID_ARG
    assert L.nvfp4_attn_workspace_size(None) == nv.NVFP4_ERR_INVALID_ARG
    assert nv.nvfp4_attn_workspace_size() > 0
    # nothing to do: no pointer is looked at
    assert L.nvfp4_attn_paged(None, cache(), batch(b=0), 1.0, None, None, None, 0, None) == nv.NVFP4_OK
    assert L.nvfp4_kv_append(None, None, None, how(), cache(), batch(tokens=0), None, None) == nv.NVFP4_OK
    assert norm(rows(), None, None, 0, 64, None, None) == nv.NVFP4_OK


def test_python_checks():
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="CUDA bfloat16"):
        nv.nvfp4_qk_norm_rope(x, None, None, None, q_out=None)
    c = torch.zeros(4, 3, 16, 64, dtype=torch.uint8)
    s = torch.ones(4, 3)
    i = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="shape mismatch"):
        nv.nvfp4_kv_append(x, x[:1], c, c, s, s, i, i[0, :3], i[0, :2], 1)
    with pytest.raises((TypeError, ValueError)):
        nv.nvfp4_attn_paged(x, c, c, s, s, i, i[0, :3], i[0, :2], 1)
