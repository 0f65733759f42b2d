"""Speculative decoding of a batch behind one shared prompt, a step from lengths to lengths.

    block tables from lengths -> qkv projection (NVFP4 GEMV) -> norm, rotation and
    append -> attention, the prompt read once for all -> output projection and
    vocabulary head (NVFP4 GEMVs) -> verification of the drafts -> new drafts

The prompt's keys and values are stored once, in pages that all sequences' tables
begin with.  A step brings a sequence's last token and its drafts; all state (lengths,
tables, pages held, the ring of free pages, tokens) stays on the device and is updated
in place, so that a step is captured once in a CUDA graph and replayed.  Weights are
random; the target is one gated attention layer of the benchmark's projections'
sizes over token embeddings, the draft model the embeddings and the head alone.

    python examples/speculative_decoding.py [--batch 32] [--prompt 4096] [--drafts 4] [--steps 32]

Prints the time of a step, the tokens that a sequence gains in one, and the largest
difference of the last step's attention from a plain fp64 computation.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import nvfp4_weight_quantized_gemv_gb300 as nv  # noqa: E402
from decode_attention import D, HIDDEN, HKV, HQ, OUT, PAGE, QKV, rope_table  # noqa: E402

VOCAB = 4096


class Server:
    def __init__(self, gen, batch, prompt, drafts, steps):
        def weight(n, k, size=0.02):
            return nv.nvfp4_quantize_bf16((torch.randn(n, k, generator=gen, device="cuda") * size).bfloat16())

        def ints(x):
            return torch.tensor(x, dtype=torch.int32, device="cuda")

        self.gen, self.batch, self.drafts, self.rows = gen, batch, drafts, batch * (drafts + 1)
        self.prompt = prompt // PAGE * PAGE
        self.embedding = torch.randn(VOCAB, HIDDEN, generator=gen, device="cuda").bfloat16()
        self.w_qkv, self.w_out, self.w_head = weight(QKV, HIDDEN), weight(HIDDEN, OUT), weight(VOCAB, HIDDEN, 0.04)
        self.longest = self.prompt + (steps + 1) * (drafts + 1)
        self.angles = rope_table(self.longest)
        # pages: the prompt's, which no sequence gives back, and a ring of the others, in any order
        shared, width = self.prompt // PAGE, -(-self.longest // PAGE)
        pages = shared + batch * (width - shared)
        order = torch.randperm(pages, generator=gen, device="cuda").int()
        self.table = torch.zeros(batch, width, dtype=torch.int32, device="cuda")
        self.table[:, :shared] = order[:shared]
        self.held, self.kept, self.free = ints([shared] * batch), ints([shared] * batch), order[shared:].clone()
        self.span = torch.tensor([0, pages - shared], device="cuda")
        self.k, self.v = (torch.zeros(pages, HKV, PAGE, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                          for _ in range(2))
        self.k_scale, self.v_scale = (torch.ones(pages, HKV, device="cuda") for _ in range(2))
        self.cache = (self.k, self.v, self.k_scale, self.v_scale)
        self.group, self.prefix = ints([0, batch]), ints([self.prompt])
        self.lens, self.new = ints([self.prompt] * batch), ints([drafts + 1] * batch)
        # the prompt, stored once
        tokens = torch.randint(0, VOCAB, (self.prompt,), generator=gen, device="cuda")
        _, _, k, v = self.project(tokens)
        nv.nvfp4_kv_append(k, v, *self.cache, self.table[:1], ints([0, self.prompt]), ints([self.prompt]), self.prompt,
                           cos_sin=self.angles, max_kv_len=self.longest)
        # tokens of the next step, a row of `ids` each, and the distributions that its drafts were drawn from
        self.ids = torch.zeros(self.rows, dtype=torch.int32, device="cuda")
        self.drawn = torch.zeros(self.rows, VOCAB, device="cuda")
        self.gained = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.draft(torch.randint(0, VOCAB, (batch,), generator=gen, device="cuda").int())

    def project(self, ids):
        y = nv.nvfp4_gemv_batched(*self.w_qkv, self.embedding[ids.long()])
        return [t.unflatten(1, (-1, D)) for t in y.split([OUT, OUT, HKV * D, HKV * D], 1)]  # q, gate, k, v

    def head(self, x):
        return torch.softmax(nv.nvfp4_gemv_batched(*self.w_head, x).float(), 1)

    def draft(self, last):
        """The next step's tokens: `last`, and drafts drawn one after the other."""
        ids, drawn = self.ids.view(self.batch, -1), self.drawn.view(self.batch, -1, VOCAB)
        ids[:, 0] = last
        for i in range(self.drafts):
            drawn[:, i] = self.head(self.embedding[ids[:, i].long()])
            noise = -torch.log(torch.rand(self.batch, VOCAB, device="cuda").clamp_min(1e-20))
            ids[:, i + 1] = (drawn[:, i] / noise).argmax(1).int()  # drawn with its probabilities

    def step(self):
        cu, lens, _, _, _, _ = nv.nvfp4_kv_tables(self.table, self.held, self.free, self.span, self.lens, self.new, PAGE,
                                                  self.rows, kept=self.kept, held_out=self.held, span_out=self.span)
        q, gate, k, v = self.project(self.ids)
        most = self.drafts + 1
        q = nv.nvfp4_kv_append(k, v, *self.cache, self.table, cu, lens, most, cos_sin=self.angles, q=q,
                               max_kv_len=self.longest)
        a = nv.nvfp4_attn_paged_shared(q, *self.cache, self.table, cu, lens, self.group, self.prefix, most,
                                       max_kv_len=self.longest, max_own_len=self.longest - self.prompt, gate=gate)
        x = self.embedding[self.ids.long()] + nv.nvfp4_gemv_batched(*self.w_out, a.flatten(1))
        _, accepted, following, left = nv.nvfp4_verify_drafts(
            self.head(x), self.ids, cu, torch.rand(self.rows, device="cuda"), torch.rand(self.batch, device="cuda"),
            draft=self.drawn, kv_lens=lens)
        self.gained += accepted + 1
        self.lens.copy_(left)
        self.draft(following)
        return lens, q, gate, a

    def plain_attention(self, q, gate, lens):
        """The definition, in fp64."""
        n, out = self.drafts + 1, torch.empty(q.shape, dtype=torch.float64, device="cuda")
        for b, kv in enumerate(lens.tolist()):
            at = self.table[b, :-(-kv // PAGE)].long()
            k, v = ((c[at].float().double() * s[at].double()[:, :, None, None]).transpose(0, 1).flatten(1, 2)[:, :kv]
                    for c, s in ((self.k, self.k_scale), (self.v, self.v_scale)))
            heads = q[b * n:(b + 1) * n].double().view(n, HKV, HQ // HKV, D)
            score = torch.einsum("nhgd,htd->nhgt", heads, k) * D ** -0.5
            hidden = torch.arange(kv, device="cuda") > torch.arange(kv - n, kv, device="cuda")[:, None]
            p = torch.softmax(score.masked_fill(hidden[:, None, None], -torch.inf), -1)
            out[b * n:(b + 1) * n] = torch.einsum("nhgt,htd->nhgd", p, v).reshape(n, HQ, D)
        return out * torch.sigmoid(gate.double())


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--batch", type=int, default=32)
    ap.add_argument("--prompt", type=int, default=4096, help="tokens that all sequences begin with (whole pages of them)")
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--steps", type=int, default=32)
    args = ap.parse_args(argv)
    server = Server(torch.Generator("cuda").manual_seed(1), args.batch, args.prompt, args.drafts, args.steps)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        server.step()  # the libraries' workspaces exist before the capture
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            lens, q, gate, a = server.step()
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        for _ in range(args.steps):
            graph.replay()
        end.record()
    torch.cuda.synchronize()
    assert nv.nvfp4_device_error() == 0
    want = server.plain_attention(q, gate, lens)
    err = ((a.double() - want).abs() / want.abs().amax(-1, keepdim=True)).max().item()
    gained = server.gained.float().mean().item() / (args.steps + 1)
    print(f"{args.batch} sequences behind {server.prompt} shared tokens, {args.drafts} drafts each: "
          f"{begin.elapsed_time(end) / args.steps * 1e3:.1f} us a step of {gained:.2f} tokens a sequence, attention within "
          f"{err:.1e} of a row's largest entry")
    return err, server


if __name__ == "__main__":
    main()
