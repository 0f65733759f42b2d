"""Block tables, slot map, positions and lengths of a step, against one request after the other on the host.

Everything is whole numbers, and every one has to be equal.
"""
from __future__ import annotations

import random

import pytest
import torch

import nvfp4_weight_quantized_gemv_gb300 as nv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    nv.build()
    yield
    assert nv.nvfp4_device_error() == 0


class State:
    """A pool of pages, what every sequence holds of it, and the definition of a step."""

    def __init__(self, batch, width, page, ring, head, free, seed=0, pad=0):
        rng = self.rng = random.Random(seed)
        self.page, self.width, self.batch = page, width, batch
        self.table = [[rng.randrange(1 << 20) for _ in range(width + pad)] for _ in range(batch)]
        self.ring = [rng.randrange(1 << 20) for _ in range(ring)]
        self.head, self.tail = head, head + free
        self.held, self.kept, self.pad = [0] * batch, None, pad

    def device(self):
        table = torch.tensor(self.table, dtype=torch.int32).view(self.batch, -1).cuda()
        return (table[:, :self.width] if self.pad else table, ints(self.held), ints(self.ring),
                torch.tensor([self.head, self.tail]).cuda())

    def step(self, kv, q, tokens):
        """(cu, lens, positions, slots), and this state after it.  Where the ring has no room for all pages given back
        none is, and self.error says so."""
        held = list(self.held)
        out, back = self._step(kv, q, tokens)
        self.error = 256 if self.tail - self.head + len(back) > len(self.ring) else 0
        if self.error:
            self.held, back = [max(a, b) for a, b in zip(held, self.held)], []
        for i, p in enumerate(back):
            self.ring[(self.tail + i) % len(self.ring)] = p
        self.head, self.tail = self.head + self.used, self.tail + len(back)
        return out

    def _step(self, kv, q, tokens):
        page, ring, free, used = self.page, len(self.ring), self.tail - self.head, 0
        kept = self.kept or [0] * self.batch
        rows = pages = 0
        cu, lens, pos, slot, back = [0], [], [], [], []
        take = [self.ring[(self.head + i) % ring] for i in range(free)]
        for b in range(self.batch):
            want = kv[b] + q[b]
            ok = kv[b] >= 0 and q[b] >= 0 and 0 <= kept[b] <= self.held[b] <= self.width and want <= self.width * page
            if ok:
                rows += q[b]
                ok = q[b] == 0 or rows <= tokens
            if ok:
                need = -(-want // page)
                pages += max(0, need - self.held[b])
                ok = need <= self.held[b] or pages <= free
            if ok:
                for i in range(self.held[b], need):
                    self.table[b][i] = take[used]
                    used += 1
                stay = max(need, kept[b])
                back += self.table[b][stay:self.held[b]]
                self.held[b] = max(need, min(self.held[b], stay))
                pos += range(kv[b], want)
                slot += [self.table[b][p // page] * page + p % page for p in range(kv[b], want)]
            cu.append(len(pos))
            lens.append(want if ok else kv[b])
        rest = tokens - len(pos)
        self.used = used
        return (cu, lens, pos + [0] * rest, slot + [-1] * rest), back


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def run(state, kv, q, tokens, in_place=False, error=0):
    table, held, ring, span = state.device()
    kept = ints(state.kept) if state.kept else None
    out = dict(held_out=held, span_out=span) if in_place else {}
    got = nv.nvfp4_kv_tables(table, held, ring, span, ints(kv), ints(q), state.page, tokens, kept=kept, **out)
    word = nv.nvfp4_device_error()
    want = state.step(kv, q, tokens)
    assert word == error | state.error
    for name, a, b in zip(("cu_q", "new_lens", "positions", "slots"), got, want):
        assert a.tolist() == b, name
    assert got[4].tolist() == state.held and got[5].tolist() == [state.head, state.tail]
    assert table.tolist() == [r[:state.width] for r in state.table] and ring.tolist() == state.ring
    if in_place:
        assert got[4].data_ptr() == held.data_ptr() and got[5].data_ptr() == span.data_ptr()
    return got


@pytest.mark.parametrize("batch,page,most_q,spare,in_place", [
    (1, 16, 1, 0, False), (3, 64, 5, 2, True), (33, 16, 40, 0, False), (257, 32, 3, 1, True), (1023, 16, 7, 0, False),
    (1025, 128, 300, 5, True), (2500, 16, 2, 0, True), (8192, 256, 4, 3, False), (5, 16, 5000, 0, True), (64, 256, 1, 1, False)])
def test_steps_of_a_growing_and_ending_batch(batch, page, most_q, spare, in_place):
    """Steps one after the other: prompts, tokens, refused drafts (shorter lengths), requests that end and begin again."""
    rng = random.Random(batch * page)
    width = -(-4 * most_q // page) + 2
    total = batch * width
    s = State(batch, width, page, ring=total + 1, head=(1 << 40) + 5, free=total + 1, seed=batch, pad=3)
    kv = [0] * batch
    for step in range(4):
        q = [0 if rng.random() < 0.1 else rng.randint(1, most_q) if step % 2 == 0 else 1 for _ in range(batch)]
        for b in range(batch):
            if rng.random() < 0.2:
                kv[b] = rng.randint(0, kv[b])  # drafts that were refused, or an end
            if rng.random() < 0.1:
                kv[b] = q[b] = 0
        got = run(s, kv, q, sum(q) + spare, in_place)
        kv = got[1].tolist()
        assert all(n >= 0 for n in kv)


def test_one_prompt_of_many_pages_and_many_tokens():
    s = State(2, 5000, 16, ring=5003, head=4999, free=5003)
    run(s, [0, 0], [79_999, 3], 80_010)
    run(s, [79_999, 3], [1, 1], 2)


def test_no_sequences_and_no_tokens():
    table, held = torch.zeros(0, 4, dtype=torch.int32).cuda(), ints([])
    span = torch.tensor([3, 5]).cuda()
    cu, lens, pos, slots, held, span_out = nv.nvfp4_kv_tables(table, held, ints([1, 2, 3]), span, held, held, 16, 3)
    assert cu.tolist() == [0] and pos.tolist() == [0] * 3 and slots.tolist() == [-1] * 3 and span_out.tolist() == [3, 5]
    s = State(3, 4, 16, 8, 0, 8)
    s.held = [1, 0, 2]
    run(s, [5, 0, 32], [0, 0, 0], 0)


@pytest.mark.parametrize("free", [0, 1, 3, 4, 6, 7, 20])
def test_pages_run_out(free):
    """Those whose pages are not free wait; those who need none go on; nothing of the waiting ones changes."""
    s = State(7, 6, 16, ring=40, head=38, free=free)
    s.held = [1, 0, 1, 2, 0, 3, 1]
    run(s, [16, 0, 3, 32, 0, 48, 16], [1, 17, 2, 1, 40, 0, 16], 100)


@pytest.mark.parametrize("tokens", [0, 1, 4, 5, 11, 12, 30])
def test_tokens_do_not_fit(tokens):
    s = State(5, 6, 16, ring=40, head=0, free=40)
    s.held = [1, 0, 0, 2, 0]
    run(s, [2, 0, 0, 5, 0], [1, 3, 0, 7, 1], tokens)


def test_pages_that_are_kept():
    s = State(5, 8, 16, ring=64, head=60, free=20)
    s.held, s.kept = [4, 4, 2, 5, 0], [2, 4, 2, 0, 0]
    run(s, [0, 0, 33, 17, 0], [0, 1, 20, 1, 16], 50)


def test_lengths_that_cannot_be_used():
    bad = 1 << 30
    for kv, q in (([-1, 3, 20], [1, 1, 1]), ([5, 3, 20], [1, -2, 1]), ([5, 129, 20], [1, 0, 1]), ([5, 100, 20], [2, 29, 1]),
                  ([bad, bad, 1], [bad, bad, 1])):
        s = State(3, 8, 16, ring=64, head=0, free=20)
        s.held = [1, 2, 2]
        run(s, kv, q, 10, error=256)
    for held, kept in (([1, 9, 2], None), ([1, -1, 2], None), ([1, 2, 2], [0, 3, 0]), ([1, 2, 2], [0, -1, 0])):
        s = State(3, 8, 16, ring=64, head=0, free=20)
        s.held, s.kept = held, kept
        run(s, [5, 17, 20], [1, 1, 1], 10, error=256)


@pytest.mark.parametrize("span", [(-1, 4), (5, 4), (0, 65), (1 << 62, (1 << 62) + 65)])
def test_a_span_that_cannot_be_used_moves_no_page(span):
    s = State(3, 8, 16, ring=64, head=0, free=0)
    s.held = [1, 2, 2]
    table, held, ring, _ = s.device()
    before = table.clone(), ring.clone()
    out = nv.nvfp4_kv_tables(table, held, ring, torch.tensor(span).cuda(), ints([5, 0, 20]), ints([1, 0, 40]), 16, 50)
    assert nv.nvfp4_device_error() == 256
    assert out[0].tolist() == [0, 1, 1, 1] and out[1].tolist() == [6, 0, 20] and out[4].tolist() == [1, 2, 2]
    assert out[5].tolist() == list(span) and torch.equal(table, before[0]) and torch.equal(ring, before[1])


def test_a_ring_without_room_leaves_pages_with_their_sequences():
    s = State(2, 8, 16, ring=4, head=0, free=3)
    s.held = [3, 1]
    table, held, ring, span = s.device()
    out = nv.nvfp4_kv_tables(table, held, ring, span, ints([0, 16]), ints([0, 5]), 16, 8)
    assert nv.nvfp4_device_error() == 256
    assert out[4].tolist() == [3, 2] and out[5].tolist() == [1, 3] and ring.tolist() == s.ring
    assert out[1].tolist() == [0, 21] and table[1, 1].item() == s.ring[0]


def test_slots_pass_32_bits():
    page = (1 << 30) - 1
    table, held = ints([[page, 0]]), ints([1])
    _, _, pos, slots, *_ = nv.nvfp4_kv_tables(table, held, ints([7]), torch.tensor([0, 1]).cuda(), ints([200]), ints([100]), 256, 100)
    assert pos.tolist() == list(range(200, 300))
    assert slots.tolist() == [page * 256 + p for p in range(200, 256)] + [7 * 256 + p for p in range(44)]


@pytest.mark.parametrize("batch", [4, 3000])
def test_a_captured_step_replays_as_lengths_grow(batch):
    """Everything in place: one graph, whose replays are the steps."""
    s = State(batch, 5, 16, ring=5 * batch, head=3, free=5 * batch)
    table, held, ring, span = s.device()
    kv, q = ints([0] * batch), ints([3] * batch)

    def step():
        return nv.nvfp4_kv_tables(table, held, ring, span, kv, q, 16, 3 * batch + 1, held_out=held, span_out=span)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
        kv.copy_(out[1])
    lens = [0] * batch
    for _ in range(12):
        graph.replay()
        torch.cuda.synchronize()
        want = s.step(lens, [3] * batch, 3 * batch + 1)
        assert [t.tolist() for t in out[:4]] == list(want)
        assert held.tolist() == s.held and span.tolist() == [s.head, s.tail] and table.tolist() == s.table
        lens = want[1]
