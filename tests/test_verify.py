"""Verification of drafted tokens against its definition, one sequence after the other in 64 bits.

Tokens and counts are whole numbers and have to be equal.  Sums are held to about 2^-48 of the total, so a random
threshold falls between two implementations' sums with a probability of some vocab * 2^-47 a sequence: 1e-9.
"""
from __future__ import annotations

import math

import pytest
import torch

import nvfp4_weight_quantized_gemv_gb300 as nv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    nv.build()
    yield
    assert nv.nvfp4_device_error() == 0


def usable(r):
    return torch.where((r > 0) & (r <= 2.0 ** 64), r, torch.zeros_like(r))


def verify64(target, draft, ids, cu, u, pick, kv):
    """(out_tokens, accepted, next, new_lens) as lists, from host tensors; -7 in rows of no sequence, and in those that
    two sequences of an unusable cu_q claim."""
    out, accepted, following, lens = [-7] * ids.numel(), [], [], []
    claims = [0] * ids.numel()
    vocab = target.shape[1]
    for b in range(pick.numel()):
        t0, t1 = int(cu[b]), int(cu[b + 1])
        if t0 < 0 or t1 <= t0 or t1 > ids.numel():
            accepted.append(0)
            following.append(-1)
            lens.append(int(kv[b]))
            continue
        claims[t0:t1] = [n + 1 for n in claims[t0:t1]]
        row = t0
        while row + 1 < t1:
            x = int(ids[row + 1])
            if not 0 <= x < vocab:
                break
            q = draft[row, x].double() if draft is not None else torch.tensor(1.0).double()
            if not bool(u[row].double() * q < target[row, x].double()):
                break
            out[row] = x
            row += 1
        p = target[row].double()
        r = p.clone()
        if row + 1 < t1:
            if draft is not None:
                r = p - draft[row].double()
            elif 0 <= int(ids[row + 1]) < vocab:
                r[int(ids[row + 1])] = 0
        r = usable(r)
        if not r.any():
            r = usable(p)
        c = torch.cumsum(r, 0)
        v = float(pick[b])
        v = v if v >= 0 else 0.0
        past = (c > v * c[-1]).nonzero()
        token = int(past[0]) if len(past) else int(r.nonzero()[-1]) if r.any() else 0
        out[row] = token
        for i in range(row + 1, t1):
            out[i] = -1
        accepted.append(row - t0)
        following.append(token)
        lens.append(int(kv[b]) - (t1 - 1 - row))
    return [-7 if n > 1 else x for x, n in zip(out, claims)], accepted, following, lens


def check(target, draft, ids, cu, u, pick, kv=None, error=0):
    dev = [None if t is None else t.cuda() for t in (target, draft, ids, cu, u, pick)]
    kv = torch.arange(pick.numel(), dtype=torch.int32) * 3 + 50 if kv is None else kv
    t, d, *rest = dev
    got = nv.nvfp4_verify_drafts(t, *rest, draft=d, kv_lens=kv.cuda())
    assert nv.nvfp4_device_error() == error
    want = verify64(target, draft, ids, cu, u, pick, kv)
    for name, a, b in zip(("accepted", "next", "new_lens"), got[1:], want[1:]):
        assert a.tolist() == b, name
    assert [x for x, w in zip(got[0].tolist(), want[0]) if w != -7] == [w for w in want[0] if w != -7]
    return got


def case(seed, drafts, vocab, given, near=0.7, sharp=2.0):
    """Distributions of a target and of a draft model that is near it, drafts drawn from the latter."""
    g = torch.Generator().manual_seed(seed)
    cu = torch.tensor([0] + [d + 1 for d in drafts]).cumsum(0).int()
    rows = int(cu[-1])
    x = torch.randn(rows, vocab, generator=g) * sharp
    target = torch.softmax(x, 1)
    q = torch.softmax(x + near * torch.randn(rows, vocab, generator=g), 1)
    drawn = torch.multinomial(q, 1, generator=g)[:, 0].int()
    ids = torch.cat([drawn[-1:], drawn[:-1]])  # row t's draft is the token of row t + 1
    return (target, q if given else None, ids, cu, torch.rand(rows, generator=g), torch.rand(len(drafts), generator=g))


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("drafts,vocab", [
    ([0], 1), ([1], 2), ([3], 5), ([4, 0, 2], 31), ([1] * 9, 257), ([40], 1000), ([5, 5, 5], 4095), ([2, 8], 4096),
    ([2, 8], 4097), ([3] * 20, 5003), ([4, 1, 0, 7], 32000), ([3, 3, 3, 3, 3], 50001), ([1] * 40, 8192), ([70, 33], 4100),
    ([6, 2], 151999)])
def test_random_distributions(drafts, vocab, given):
    for seed in range(3):
        check(*case(seed + vocab, drafts, vocab, given))


@pytest.mark.parametrize("vocab", [777, 9001])
@pytest.mark.parametrize("offset,stride", [(0, 0), (1, 3), (2, 8), (3, 1)])
def test_rows_of_any_alignment(vocab, offset, stride):
    """Rows inside a larger array, the two distributions on equal and on different 16-byte phases."""
    target, draft, *rest = case(5, [3, 4, 2], vocab, True)
    rows = target.shape[0]

    def inside(x, off, pad):
        big = torch.full((rows, vocab + off + pad), math.nan)
        big[:, off:off + vocab] = x
        return big.cuda()[:, off:off + vocab]

    want = verify64(target, draft, *rest, torch.zeros(3, dtype=torch.int32))
    for t, d in ((inside(target, offset, stride), inside(draft, offset, stride)), (inside(target, offset, stride), draft.cuda()),
                 (target.cuda(), inside(draft, offset, stride))):
        got = nv.nvfp4_verify_drafts(t, *(x.cuda() for x in rest), draft=d)
        assert got[3] is None
        assert [x.tolist() for x in got[:3]] == list(want[:3])


@pytest.mark.parametrize("vocab", [16, 64, 8192, 65536])
def test_thresholds_on_a_boundary(vocab):
    """Equal weights of a power of two: cumulative sums are exact, and a threshold that meets one goes to the next."""
    b = 33
    target = torch.full((b, vocab), 1.0 / vocab)
    pick = (torch.arange(b) * (vocab // 16) % vocab).float() / vocab
    pick[-1] = 1 - 2.0 ** -24
    cu = torch.arange(b + 1, dtype=torch.int32)
    got = check(target, None, torch.zeros(b, dtype=torch.int32), cu, torch.zeros(b), pick)
    assert got[2].tolist()[:-1] == (torch.arange(b - 1) * (vocab // 16) % vocab).tolist()
    assert got[2].tolist()[-1] == vocab - 1


def test_acceptance_on_its_boundary():
    """u q(x) < p(x) is decided exactly: u q is not rounded."""
    vocab = 8
    # products: (1 - 2^-24)^2 = p + 2^-48; p; p (as 0.25 + 2^-26 rounds to 0.25); 0; 0 < 2^-149; p; and
    # 0.5 (1 + 2^-22) (1 - 2^-23) = 0.5 (1 + 2^-23 - 2^-45), below p by less than half a step; p - 2^-24 + 2^-48
    u = torch.tensor([1 - 2.0 ** -24, 0.5, 0.5, 0.0, 0.0, 2.0 ** -24, 1 - 2.0 ** -23, 1 - 2.0 ** -24])
    q = torch.tensor([1 - 2.0 ** -24, 0.5, 0.5, 0.5, 0.0, 0.25, 0.5 * (1 + 2.0 ** -22), 1 - 2.0 ** -24])
    p = torch.tensor([1 - 2.0 ** -23, 0.25, 0.25 + 2.0 ** -26, 0.0, 2.0 ** -149, 2.0 ** -26, 0.5 * (1 + 2.0 ** -23),
                      1 - 2.0 ** -24])
    rows = 2 * len(u)
    target, draft = torch.full((rows, vocab), 0.01), torch.full((rows, vocab), 0.01)
    target[::2, 3], draft[::2, 3] = p, q
    ids = torch.full((rows,), 3, dtype=torch.int32)
    cu = torch.arange(0, rows + 1, 2, dtype=torch.int32)
    got = check(target, draft, ids, cu, u.repeat_interleave(2), torch.full((len(u),), 0.3))
    assert got[1].tolist() == [0, 0, 0, 0, 1, 0, 1, 1]


def test_a_draft_model_that_is_the_target():
    """p == q: every draft with a probability is accepted (u < 1)."""
    target, _, ids, cu, u, pick = case(3, [6, 6], 6000, True, near=0.0)
    assert check(target, target.clone(), ids, cu, u, pick)[1].tolist() == [6, 6]


@pytest.mark.parametrize("vocab", [100, 10000])
def test_a_refused_draft_where_p_is_nowhere_above_q(vocab):
    """The residual is empty: the next token comes from p itself."""
    target, draft, ids, cu, u, pick = case(4, [2, 1], vocab, True)
    check(target * 0.5, torch.maximum(target, draft) * 2, ids, cu, torch.full_like(u, 0.9999), pick)


@pytest.mark.parametrize("vocab", [50, 7000])
def test_a_draft_that_has_all_the_weight(vocab):
    """One-hot targets (greedy decoding) against drafts without probabilities."""
    g = torch.Generator().manual_seed(1)
    best = torch.randint(0, vocab, (12,), generator=g)
    target = torch.nn.functional.one_hot(best, vocab).float()
    ids = torch.cat([torch.zeros(1), best[:-1]]).int()
    ids[5] = (ids[5] + 1) % vocab
    cu = torch.tensor([0, 4, 8, 12], dtype=torch.int32)
    got = check(target, None, ids, cu, torch.rand(12, generator=g), torch.rand(3, generator=g))
    assert got[1].tolist() == [3, 0, 3] and got[2].tolist() == [int(best[3]), int(best[4]), int(best[11])]


@pytest.mark.parametrize("vocab", [60, 9000])
def test_entries_that_are_no_weights(vocab):
    """NaN, infinite, negative and denormal entries, and a row that has none left."""
    target, draft, ids, cu, u, pick = case(6, [1, 0, 1, 0], vocab, True)
    target[:, 3], target[:, 5], target[:, 7], target[:, 9], target[:, 11] = math.nan, math.inf, -1.0, 2.0 ** -140, 2.0 ** 65
    draft[:, 13], draft[:, 15], draft[:, 17] = math.nan, math.inf, -0.5
    ids[:] = 20
    check(target, draft, ids, cu, torch.ones_like(u), pick)
    target[2:4] = 0
    target[4] = math.nan
    got = check(target, draft, ids, cu, torch.ones_like(u), torch.zeros(4), error=256)
    assert got[2].tolist()[1:3] == [0, 17]  # row 2 has no weight; row 3 has 0 - (-0.5) at entry 17


def test_random_numbers_out_of_their_range():
    target, draft, ids, cu, u, _ = case(7, [2, 2, 2, 2], 5000, True)
    target[:, -7:] = 0
    pick = torch.tensor([1.0, 5.0, -1.0, math.nan])
    got = check(target, draft, ids, cu, torch.zeros_like(u), pick)  # u = 0: all are accepted
    assert got[1].tolist() == [2] * 4 and got[2].tolist() == [4992, 4992, 0, 0]
    check(target, draft, ids, cu, torch.full_like(u, math.nan), pick)


def test_tokens_outside_the_vocabulary_and_unusable_rows():
    target, draft, ids, cu, u, pick = case(8, [2, 2, 2], 4500, True)
    ids[1], ids[4], ids[8] = -1, 4500, 1 << 30
    check(target, draft, ids, cu, torch.zeros_like(u), pick, error=256)
    check(target, None, ids, cu, torch.zeros_like(u), pick, error=256)
    target, draft, ids, _, u, pick = case(8, [2, 2, 2], 300, True)
    for bad in ([0, 4, 3, 9], [0, 3, 10, 9], [-1, 3, 6, 9], [0, 0, 5, 5]):
        cu = torch.tensor(bad, dtype=torch.int32)
        check(target, draft, ids, cu, u, pick, error=0 if bad[1] == 0 else 256)


def test_rows_of_no_sequence_stay():
    target, draft, ids, cu, u, pick = (t.cuda() for t in case(9, [2, 3], 600, True))
    import ctypes
    out = torch.full((7,), 99, dtype=torch.int32, device="cuda")
    small = torch.full((4, 2), 99, dtype=torch.int32, device="cuda")
    rows = nv.nvfp4_draft_rows(target.data_ptr(), draft.data_ptr(), 600, 600, ids.data_ptr(), 7, 600)
    cu = torch.tensor([1, 3, 5], dtype=torch.int32, device="cuda")
    nv._check(nv.lib().nvfp4_verify_drafts(rows, cu.data_ptr(), None, u.data_ptr(), pick.data_ptr(), 2, out.data_ptr(),
                                           small[0].data_ptr(), small[1].data_ptr(), None,
                                           ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)))
    torch.cuda.synchronize()
    assert out[[0, 5, 6]].tolist() == [99] * 3 and (out[1:5] != 99).all() and (small[2:] == 99).all()


def test_no_sequences():
    t = torch.zeros(0, 50, device="cuda")
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    got = nv.nvfp4_verify_drafts(t, z, torch.zeros(1, dtype=torch.int32, device="cuda"), t[:, 0], t[:, 0], kv_lens=z)
    assert [x.numel() for x in got] == [0, 0, 0, 0]


def test_tokens_are_distributed_as_the_targets():
    """Every token's share of 300000 first tokens: chi-square of 11 live tokens below its 1 - 1e-6 quantile (48)."""
    g = torch.Generator().manual_seed(3)
    n, vocab = 300000, 12
    p = torch.tensor([0.3, 0.02, 0.1, 0.05, 0.13, 0.0, 0.08, 0.02, 0.1, 0.05, 0.05, 0.1])
    q = torch.tensor([0.1, 0.1, 0.05, 0.05, 0.2, 0.1, 0.02, 0.08, 0.05, 0.1, 0.1, 0.05])
    count = torch.zeros(vocab, dtype=torch.int64)
    batch = 30000
    for _ in range(n // batch):
        x = torch.multinomial(q, batch, replacement=True, generator=g).int()
        ids = torch.stack([torch.zeros_like(x), x], 1).flatten()
        cu = torch.arange(0, 2 * batch + 1, 2, dtype=torch.int32)
        u, pick = torch.rand(2 * batch, generator=g), torch.rand(batch, generator=g)
        rows = [t.expand(2 * batch, vocab).contiguous().cuda() for t in (p, q)]
        out = nv.nvfp4_verify_drafts(rows[0], ids.cuda(), cu.cuda(), u.cuda(), pick.cuda(), draft=rows[1])
        count += torch.bincount(out[0].cpu()[::2], minlength=vocab)
    want = p.double() * n
    assert count[5] == 0
    live = want > 0
    assert float(((count - want)[live] ** 2 / want[live]).sum()) < 48


def test_same_tokens_every_time_and_in_a_graph():
    target, draft, ids, cu, u, pick = (t.cuda() for t in case(11, [5] * 30, 20011, True))
    kv = torch.full((30,), 100, dtype=torch.int32, device="cuda")
    want = nv.nvfp4_verify_drafts(target, ids, cu, u, pick, draft=draft, kv_lens=kv)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = nv.nvfp4_verify_drafts(target, ids, cu, u, pick, draft=draft, kv_lens=kv)
    for _ in range(5):
        for t in got:
            t.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
