"""One gated attention layer of a served model, from hidden states to hidden states.

    qkv projection (NVFP4 GEMV) -> norm, rotation and append to the paged 8-bit
    cache -> attention over the cache, gated -> output projection (NVFP4 GEMV)

First a ragged batch of prompts in one call of each operator, then decode steps
of one token a sequence, captured once in a CUDA graph and replayed while the
lengths grow on the device.  Weights and hidden states are random; the layer's
sizes are those of the benchmark's projections (qkv 14336 x 5120: 24 query
heads with their gates and 4 kv heads of 256; o_proj 5120 x 6144).

    python examples/decode_attention.py [--batch 8] [--prompt 700] [--steps 64]

Prints the time of a step and the largest difference of the last step's
attention from a plain fp64 computation over the cache's contents.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_weight_quantized_gemv_gb300 as nv  # noqa: E402

HIDDEN, HQ, HKV, D, ROT, PAGE = 5120, 24, 4, 256, 64, 64
QKV, OUT = (2 * HQ + 2 * HKV) * D, HQ * D


def rope_table(positions, theta=10000.0):
    angle = torch.arange(positions).double()[:, None] * theta ** (-torch.arange(ROT // 2).double() / (ROT // 2))
    return torch.cat([angle.cos(), angle.sin()], 1).float().cuda()


class Layer:
    def __init__(self, gen, batch, longest):
        def weight(n, k):
            return nv.nvfp4_quantize_bf16((torch.randn(n, k, generator=gen, device="cuda") * 0.02).bfloat16())

        def norm():
            return (1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).bfloat16()

        self.w_qkv, self.w_out, self.q_norm, self.k_norm = weight(QKV, HIDDEN), weight(HIDDEN, OUT), norm(), norm()
        self.table = rope_table(longest)
        per = -(-longest // PAGE)  # pages of a sequence, in any order in the cache
        self.pages = torch.randperm(batch * per, generator=gen, device="cuda").int().view(batch, per)
        self.k, self.v = (torch.zeros(batch * per, HKV, PAGE, D, dtype=torch.uint8, device="cuda")
                          .view(torch.float8_e4m3fn) for _ in range(2))
        self.k_scale, self.v_scale = (torch.ones(batch * per, HKV, device="cuda") for _ in range(2))

    def cache(self):
        return self.k, self.v, self.k_scale, self.v_scale, self.pages

    def forward(self, x, cu_q, kv_lens, max_q_len, max_kv_len):
        """x bf16 [tokens, HIDDEN] -> (bf16 [tokens, HIDDEN], the queries and gates that attention read)."""
        y = nv.nvfp4_gemv_batched(*self.w_qkv, x)
        q, gate, k, v = (t.unflatten(1, (-1, D)) for t in y.split([OUT, OUT, HKV * D, HKV * D], 1))  # views
        batch = (cu_q, kv_lens, max_q_len)
        q = nv.nvfp4_kv_append(k, v, *self.cache(), *batch, cos_sin=self.table, k_weight=self.k_norm, q=q,
                               q_weight=self.q_norm, max_kv_len=max_kv_len)
        a = nv.nvfp4_attn_paged(q, *self.cache(), *batch, max_kv_len=max_kv_len, gate=gate)
        return nv.nvfp4_gemv_batched(*self.w_out, a.flatten(1)), q, gate, a


def plain_attention(layer, q, gate, kv_lens):
    """The definition, in fp64, for one token a sequence."""
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(kv_lens.tolist()):
        at = layer.pages[b, :-(-n // PAGE)].long()
        k, v = ((c[at].float().double() * s[at].double()[:, :, None, None]).transpose(0, 1).flatten(1, 2)[:, :n]
                for c, s in ((layer.k, layer.k_scale), (layer.v, layer.v_scale)))
        heads = q[b].double().view(HKV, HQ // HKV, D)
        p = torch.softmax(heads @ k.transpose(1, 2) * D ** -0.5, -1)
        out[b] = (p @ v).view(HQ, D)
    return out * torch.sigmoid(gate.double())


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=700, help="longest prompt; the others are shorter")
    ap.add_argument("--steps", type=int, default=64)
    args = ap.parse_args(argv)
    gen = torch.Generator("cuda").manual_seed(1)
    longest = args.prompt + args.steps + 3
    layer = Layer(gen, args.batch, longest)

    lens = [max(1, args.prompt - 37 * b % args.prompt) for b in range(args.batch)]
    cu = torch.tensor([0] + lens).cumsum(0).int().cuda()
    kv_lens = torch.tensor(lens).int().cuda()
    x = torch.randn(sum(lens), HIDDEN, generator=gen, device="cuda").bfloat16()
    layer.forward(x, cu, kv_lens, max(lens), longest)

    cu = torch.arange(args.batch + 1).int().cuda()
    x = torch.randn(args.batch, HIDDEN, generator=gen, device="cuda").bfloat16()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        kv_lens += 1
        layer.forward(x, cu, kv_lens, 1, longest)  # the library's workspaces exist before the capture
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            kv_lens += 1
            y, q, gate, a = layer.forward(x, cu, kv_lens, 1, longest)
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        graph.replay()
        begin.record()
        for _ in range(args.steps):
            graph.replay()
        end.record()
    torch.cuda.synchronize()
    assert nv.nvfp4_device_error() == 0
    want = plain_attention(layer, q, gate, kv_lens)
    err = ((a.double() - want).abs() / want.abs().amax(-1, keepdim=True)).max().item()
    print(f"{args.batch} sequences of {min(lens)} to {max(lens)} tokens and {args.steps + 2} more: "
          f"{begin.elapsed_time(end) / args.steps * 1e3:.1f} us a step, attention within {err:.1e} of a row's largest entry")
    return err, y


if __name__ == "__main__":
    main()
