"""Outputs that a call allocates belong to the stream that the call is given.

PyTorch's allocator orders a block's uses by the stream it was allocated on: an
output from another stream's memory could still be read there, or be given away
again, while the call writes it.  Which memory an output is made of shows in its
address: a block just freed on a stream is what the next allocation of that size
on it gets.
"""
from __future__ import annotations

import pytest
import torch

import nvfp4_weight_quantized_gemv_gb300 as nv
from test_attention_ops import Paged, built, randn, table  # noqa: F401

pytestmark = pytest.mark.gpu


def freed(like, stream):
    """The address of a block of like's size that was allocated on `stream` and given back."""
    with torch.cuda.stream(stream):
        t = torch.empty_like(like)
        at = t.data_ptr()
        del t
    return at


def check(call, stream):
    """call(stream) -> outputs, of memory of `stream` and right there."""
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    for handle in (stream, stream.cuda_stream):
        for i, like in enumerate(want):
            here, there = freed(like, torch.cuda.current_stream()), freed(like, stream)
            got = call(handle)
            at = [t.data_ptr() for t in got]
            assert here not in at and there in at, i
            with torch.cuda.stream(stream):
                assert all(torch.equal(a, b) for a, b in zip(got, want))
            del got
    assert torch.cuda.current_stream() == torch.cuda.default_stream()



def test_norm_rope_allocates_on_its_stream():
    g = torch.Generator().manual_seed(1)
    q, k = randn(g, 16384, 4, 256).bfloat16().cuda(), randn(g, 16384, 2, 256).bfloat16().cuda()
    pos, cs = torch.arange(16384, dtype=torch.int32).cuda(), table(16384, 64).cuda()
    check(lambda s: nv.nvfp4_qk_norm_rope(q, k, pos, cs, stream=s), torch.cuda.Stream())


def test_append_and_attention_allocate_on_their_stream():
    p = Paged(3, [4096], [4096], 1, 128, 64)
    q, kv = randn(p.g, 4096, 32, 128).bfloat16().cuda(), randn(p.g, 4096, 1, 128).bfloat16().cuda()
    side = torch.cuda.Stream()
    check(lambda s: [nv.nvfp4_kv_append(kv, kv, *p.args(), 4096, q=q, stream=s)], side)
    check(lambda s: [nv.nvfp4_attn_paged(q, *p.args(), 4096, stream=s)], side)
    assert nv.nvfp4_device_error() == 0


def test_gemv_quantizer_ffn_and_experts_allocate_on_their_stream():
    g = torch.Generator().manual_seed(2)
    n, k = 4096, 2048
    w, x = randn(g, n, k).bfloat16().cuda(), randn(g, 512, k).bfloat16().cuda()
    side = torch.cuda.Stream()
    check(lambda s: nv.nvfp4_quantize(w, stream=s)[:2], side)
    w4, down = nv.nvfp4_quantize(w), nv.nvfp4_quantize(randn(g, k, n // 2).bfloat16().cuda())
    check(lambda s: [nv.nvfp4_gemv_batched(*w4, x, stream=s)], side)
    check(lambda s: [nv.nvfp4_gemv_batched_ex(*w4, x, stream=s)], side)
    check(lambda s: [nv.nvfp4_gemv_swiglu(*w4, x, stream=s)], side)
    h = torch.empty(512, n // 2, dtype=torch.bfloat16, device="cuda")  # else it takes the block that y is looked for in
    check(lambda s: [nv.nvfp4_ffn_swiglu(w4, down, x, h=h, stream=s)], side)
    experts = [t[None] for t in w4[:2]] + [w4[2]]
    of = torch.tensor([0, 512], dtype=torch.int32).cuda()
    token = torch.arange(512, dtype=torch.int32).cuda()
    check(lambda s: [nv.nvfp4_moe_gemv_grouped(*experts, x, of, token, stream=s)], side)
    assert nv.nvfp4_device_error() == 0


class Elsewhere(torch.Tensor):
    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError


def test_tensors_of_another_device_are_refused():
    """Tensors that say they are on a second GPU (and have no memory): each argument alone, and all of them."""
    p = Paged(3, [4], [40], 1, 128, 64)
    q, kv = randn(p.g, 4, 2, 128).bfloat16().cuda(), randn(p.g, 4, 1, 128).bfloat16().cuda()
    pos, cs, w = torch.arange(4, dtype=torch.int32).cuda(), table(64, 64).cuda(), torch.ones(128).bfloat16().cuda()
    ws = torch.empty(nv.nvfp4_attn_workspace_size(), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)

    def norm(q, k, pos, cs, qw, kw, q_out, k_out):
        nv.nvfp4_qk_norm_rope(q, k, pos, cs, qw, kw, q_out=q_out, k_out=k_out)

    def append(k, v, kc, vc, ks, vs, table_, cu, lens, cs, kw, q, qw, q_out):
        nv.nvfp4_kv_append(k, v, kc, vc, ks, vs, table_, cu, lens, 4, cs, kw, q, qw, q_out=q_out, max_kv_len=40)

    def attend(q, kc, vc, ks, vs, table_, cu, lens, gate, out, ws):
        nv.nvfp4_attn_paged(q, kc, vc, ks, vs, table_, cu, lens, 4, 40, gate=gate, out=out, workspace=ws)

    def other(t):
        return Elsewhere._make_wrapper_subclass(Elsewhere, t.size(), t.stride(), dtype=t.dtype, device=torch.device("cuda:1"))

    for call, args in ((norm, [q, kv, pos, cs, w, w, out, torch.empty_like(kv)]),
                       (append, [kv, kv, *p.args(), cs, w, q, w, out]), (attend, [q, *p.args(), q, out, ws])):
        call(*args)
        for i in range(len(args)):
            with pytest.raises(ValueError, match="is on cuda:1, the current device is cuda:0"):
                call(*args[:i], other(args[i]), *args[i + 1:])
        with pytest.raises(ValueError, match="is on cuda:1, the current device is cuda:0"):
            call(*[other(t) for t in args])
    assert nv.nvfp4_device_error() == 0


def test_the_default_stream_by_object_and_by_handle():
    """Handle 0 is the default stream, also where another one is current."""
    g = torch.Generator().manual_seed(4)
    w, q = randn(g, 4096, 1024).bfloat16().cuda(), randn(g, 8192, 4, 128).bfloat16().cuda()
    w4 = nv.nvfp4_quantize(w)
    x = randn(g, 512, 1024).bfloat16().cuda()
    side, default = torch.cuda.Stream(), torch.cuda.default_stream()
    for call in (lambda s: nv.nvfp4_qk_norm_rope(q, None, None, None, stream=s)[0], lambda s: nv.nvfp4_gemv_batched(*w4, x, stream=s)):
        want = call(None)
        torch.cuda.synchronize()
        for handle in (default, 0):
            there = freed(want, default)
            with torch.cuda.stream(side):
                got = call(handle)
                assert torch.cuda.current_stream() == side
            assert got.data_ptr() == there
            assert torch.equal(got, want)
            del got
