"""The operators around a batch of requests together, as a server uses them.

A prompt that all requests begin with is stored once; every step brings each request's last token and its drafts:

    tables -> append -> attention behind the shared prefix -> (a stand-in for the rest of the model) -> verification

and the verified lengths are the next step's.  Every operator is checked against its definition, on what the ones
before it left on the GPU.
"""
from __future__ import annotations

import pytest
import torch

import nvfp4_weight_quantized_gemv_gb300 as nv
from test_attention_ops import F64, attn64, built, close_bf16, e4m3_64, heads64, need64, randn, table  # noqa: F401
from test_kv_tables import State
from test_verify import verify64

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Server:
    def __init__(self, seed, batch, prefix, page, hq, hkv, d, vocab, width=None):
        g = self.g = torch.Generator().manual_seed(seed)
        self.batch, self.prefix, self.page, self.hq, self.hkv, self.d, self.vocab = batch, prefix, page, hq, hkv, d, vocab
        shared = prefix // page
        # rows of the table wide enough for a bound on lengths that allows for sharing
        self.width = width or -(-110_000_000 // ((batch - 3) * hkv * 2 * d * page))
        pages = shared + batch * 8
        self.k, self.v = (torch.zeros(pages, hkv, page, d, dtype=torch.uint8).cuda().view(torch.float8_e4m3fn) for _ in range(2))
        self.ks, self.vs = torch.ones(pages, hkv).cuda(), torch.ones(pages, hkv).cuda()
        order = torch.randperm(pages, generator=g).int()
        self.table = torch.zeros(batch, self.width, dtype=torch.int32)
        self.table[:, :shared] = order[:shared]
        self.table = self.table.cuda()
        self.held = ints([shared] * batch)
        self.kept = ints([shared] * batch)
        self.ring = order[shared:].cuda()
        self.span = torch.tensor([0, pages - shared]).cuda()
        self.lens = ints([prefix] * batch)
        self.cos_sin = table(prefix + 8 * page, d).cuda()
        self.head = (randn(g, hq * d, vocab) * (hq * d) ** -0.5 * 40).cuda()
        # the prompt itself, stored once
        k, v = (randn(g, prefix, hkv, d).bfloat16().cuda() for _ in range(2))
        nv.nvfp4_kv_append(k, v, *self.cache(), self.table[:1], ints([0, prefix]), ints([prefix]), prefix,
                           cos_sin=self.cos_sin, max_kv_len=prefix)

    def cache(self):
        return self.k, self.v, self.ks, self.vs

    def step(self, x, ids, draft, u, pick, new, most):
        """x bf16 [rows, hq + 2 hkv, d]; `new` tokens a request; returns everything that the operators gave."""
        rows = x.shape[0]
        cu, lens, positions, slots, _, _ = out = nv.nvfp4_kv_tables(
            self.table, self.held, self.ring, self.span, self.lens, new, self.page, rows, kept=self.kept,
            held_out=self.held, span_out=self.span)
        q, k, v = x.split([self.hq, self.hkv, self.hkv], 1)
        q = nv.nvfp4_kv_append(k, v, *self.cache(), self.table, cu, lens, most, cos_sin=self.cos_sin, q=q,
                               max_kv_len=self.cos_sin.shape[0])
        y = nv.nvfp4_attn_paged_shared(q, *self.cache(), self.table, cu, lens, self.group, self.prefixes, most)
        target = torch.softmax(y.flatten(1).float() @ self.head, 1)
        verified = nv.nvfp4_verify_drafts(target, ids, cu, u, pick, draft=draft, kv_lens=lens)
        self.lens.copy_(verified[3])
        return out, q, y, target, verified


@pytest.mark.parametrize("batch,page,hq,hkv,d", [(5, 16, 8, 2, 64), (4, 64, 6, 1, 128), (9, 32, 24, 4, 256)])
def test_steps_of_a_batch_behind_a_shared_prompt(batch, page, hq, hkv, d):
    s = Server(batch, batch, 256, page, hq, hkv, d, 3001)
    s.group, s.prefixes = ints([0, batch]), ints([256])
    state = State(batch, s.width, page, len(s.ring), 0, len(s.ring))
    state.held, state.kept = s.held.tolist(), s.kept.tolist()
    state.ring, state.table = s.ring.tolist(), s.table.tolist()
    g = s.g
    for turn in range(4):
        new = [1 + (turn + b) % 4 for b in range(batch)]
        if turn == 3:
            new[0] = 0  # waits this turn
        rows = sum(new)
        x = randn(g, rows, hq + 2 * hkv, d).bfloat16().cuda()
        draft = torch.softmax(2 * randn(g, rows, s.vocab), 1).cuda()
        ids = torch.multinomial(draft.cpu(), 1, generator=g)[:, 0].int().cuda()
        u, pick = torch.rand(rows, generator=g).cuda() * 0.2, torch.rand(batch, generator=g).cuda()
        before = s.lens.tolist()
        (cu, lens, positions, slots, _, _), q, y, target, (out, accepted, following, left) = s.step(
            x, ids, draft, u, pick, ints(new), max(new))
        assert nv.nvfp4_device_error() == 0
        # tables
        want = state.step(before, new, rows)
        assert [t.tolist() for t in (cu, lens, positions, slots)] == list(want)
        assert s.table.tolist() == state.table and s.held.tolist() == state.held
        # queries and keys: rotated at the positions, values at the slots
        at = s.cos_sin.cpu()[positions.cpu().long()]
        close_bf16(q, heads64(x[:, :hq].cpu(), None, at, d, False), 2.0 ** -20)
        page_of, slot_of = slots.cpu() // page, slots.cpu() % page
        stored = s.v.cpu().float()[page_of, :, slot_of] * s.vs.cpu()[page_of][..., None]
        far = (stored - x[:, hq + hkv:].cpu().float()).abs()  # half a step of E4M3: 2^-4 of the value, 2^-10 of the scale
        assert (far <= 2.0 ** -4 * stored.abs() + 2.0 ** -10 * s.vs.cpu()[page_of][..., None]).all()
        # attention over the pages that the tables name
        s.qs, s.kvs, s.cu = new, lens.tolist(), cu.cpu()
        view = type("View", (), dict(qs=new, kvs=lens.tolist(), cu=cu.cpu(), page=page, hkv=hkv, d=d, table=s.table.cpu(),
                                     host=lambda self: [s.k.cpu().float().to(F64), s.v.cpu().float().to(F64), s.ks.cpu().to(F64),
                                                        s.vs.cpu().to(F64)]))()
        ref, size = attn64(view, q.cpu(), d ** -0.5)
        close_bf16(y, ref, 2.0 ** -8 * size)
        # verification
        want = verify64(target.cpu(), draft.cpu(), ids.cpu(), cu.cpu(), u.cpu(), pick.cpu(), lens.cpu())
        assert [t.tolist() for t in (out, accepted, following, left)] == list(want)
        assert all(n >= b + (m > 0) for n, b, m in zip(s.lens.tolist(), before, new))
    # all requests end: what they hold beyond the prompt is given back
    s.lens.zero_()
    nv.nvfp4_kv_tables(s.table, s.held, s.ring, s.span, s.lens, ints([0] * batch), page, 0, kept=s.kept, held_out=s.held,
                       span_out=s.span)
    assert s.held.tolist() == s.kept.tolist()
    free = int(s.span[1] - s.span[0])
    assert free == len(s.ring)
    assert sorted(s.ring.tolist()) == sorted(set(range(len(s.ring) + 256 // page)) - set(s.table[0, :256 // page].tolist()))


def test_a_captured_step_replays():
    """The same step from a graph: all state in place, random numbers and tokens copied in."""
    runs = []
    for captured in (False, True):
        batch, n = 4, 3
        s = Server(7, batch, 128, 16, 8, 2, 64, 500)
        s.group, s.prefixes = ints([0, batch]), ints([128])
        g, rows = s.g, batch * n
        x = torch.zeros(rows, 12, 64, dtype=torch.bfloat16, device="cuda")
        ids, draft = ints([0] * rows), torch.zeros(rows, 500, device="cuda")
        u, pick, new = torch.zeros(rows, device="cuda"), torch.zeros(batch, device="cuda"), ints([n] * batch)
        args = (x, ids, draft, u, pick, new, n)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        if captured:
            s.step(*args)  # workspaces and libraries are set up
            torch.cuda.synchronize()
            s = Server(7, batch, 128, 16, 8, 2, 64, 500)
            s.group, s.prefixes = ints([0, batch]), ints([128])
            with torch.cuda.graph(graph, stream=stream):
                out = s.step(*args)
        g, all_out = torch.Generator().manual_seed(5), []
        for _ in range(5):
            x.copy_(randn(g, rows, 12, 64).bfloat16())
            draft.copy_(torch.softmax(randn(g, rows, 500), 1))
            ids.copy_(torch.multinomial(draft.cpu(), 1, generator=g)[:, 0])
            u.copy_(torch.rand(rows, generator=g) * 0.3)
            pick.copy_(torch.rand(batch, generator=g))
            if captured:
                graph.replay()
            else:
                out = s.step(*args)
            torch.cuda.synchronize()
            (cu, lens, pos, slots, _, _), _, y, _, verified = out
            all_out += [t.clone() for t in (cu, lens, pos, slots, y, *verified, s.lens, s.held, s.span, s.ring, s.table)]
        assert nv.nvfp4_device_error() == 0
        runs.append(all_out)
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_example_runs(capsys):
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import speculative_decoding
    err, s = speculative_decoding.main(["--batch", "7", "--prompt", "400", "--drafts", "3", "--steps", "6"])
    assert err < 2.0 ** -7
    lens, gained = s.lens.tolist(), s.gained.tolist()
    assert lens == [384 + n for n in gained] and all(7 <= n <= 28 for n in gained)
    assert all(h >= -(-n // 64) for h, n in zip(s.held.tolist(), lens))
    assert len(set(s.table[:, :6].flatten().tolist())) == 6
    assert "us a step" in capsys.readouterr().out
