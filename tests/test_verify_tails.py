"""Rows of which whole parts have no weight: the next token always has some.

Vocabularies padded to a multiple of something end in entries without weight, and masks leave whole ranges without; the
parts that a row is shared out in are then empty.  Tokens have to be the definition's: at u_next of 1 and more the last
entry with a weight, however small it is beside the others; below that the smallest index whose cumulative sum (in 64 bits)
exceeds the threshold.  The sums are off by some 2^-46 of the total: thresholds within 2^-44 of a sum may go to either side, but
to an entry with a weight.
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


def next_tokens(target, pick, draft=None):
    """A sequence a row, or two rows whose draft is refused."""
    n, vocab = target.shape
    step = 1 if draft is None else 2
    ids = torch.zeros(step * n, dtype=torch.int32)
    if draft is not None:
        ids[1::2] = (draft >= target).int().argmax(1)
        target, draft = [torch.stack([t, torch.zeros_like(t)], 1).flatten(0, 1) for t in (target, draft)]
    got = nv.nvfp4_verify_drafts(target.cuda(), ids.cuda(), torch.arange(0, step * n + 1, step, dtype=torch.int32).cuda(),
                                 torch.ones(step * n).cuda(), pick.cuda(), draft=None if draft is None else draft.cuda())
    assert got[1].tolist() == [0] * n
    return got[2].tolist()


def empty_parts(kind, vocab):
    keep = torch.ones(vocab, dtype=torch.bool)
    if kind == "tail":
        keep[vocab - vocab // 8:] = False
    elif kind == "half":
        keep[vocab // 2:] = False
    elif kind == "head":
        keep[:vocab // 3] = False
    elif kind == "stripes":
        keep[:] = (torch.arange(vocab) * 16 // vocab) % 2 == 0
    else:  # few entries
        keep[:] = False
        keep[[vocab // 5, vocab // 2, vocab // 2 + 1]] = True
    return keep


@pytest.mark.parametrize("kind", ["tail", "half", "head", "stripes", "few"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("vocab", [2000, 8000, 8192, 30001, 131072])
def test_parts_without_weight(vocab, residual, kind):
    g = torch.Generator().manual_seed(vocab)
    n = 48
    keep = empty_parts(kind, vocab)
    x = torch.randn(n, vocab, generator=g) * 2
    target = torch.softmax(x.masked_fill(~keep, -math.inf), 1)
    draft = torch.softmax(x + torch.randn(n, vocab, generator=g), 1).masked_fill(~keep, 0.0) if residual else None
    r = target.double() if draft is None else (target.double() - draft.double()).clamp(min=0)
    if kind == "few" and residual:
        draft = target * 0.5
        draft[:, vocab // 2 + 1] = 1.0
        r = (target.double() - draft.double()).clamp(min=0)
    last = [int(row.nonzero()[-1]) for row in r]
    for u in (1.0, 1.5, math.inf):
        assert next_tokens(target, torch.full((n,), u), draft) == last
    sums = r.cumsum(1)
    for pick in (torch.full((n,), 1 - 2.0 ** -24), torch.rand(n, generator=g), torch.zeros(n)):
        at = pick.double() * sums[:, -1]
        far = (sums - at[:, None]).abs().amin(1) / sums[:, -1]
        want = [int((s > t).nonzero()[0]) for s, t in zip(sums, at)]
        got = next_tokens(target, pick, draft)
        sure = ((far > 2.0 ** -44) | (pick == 0)).tolist()
        assert [t for t, s in zip(got, sure) if s] == [t for t, s in zip(want, sure) if s]
        assert all(r[i, t] > 0 for i, t in enumerate(got))


@pytest.mark.parametrize("vocab", [8000, 131072])
def test_the_last_weight_however_small(vocab):
    """A tail of 2^-100 beside a softmax: below any sum's last bit, and still the last entry with a weight."""
    n = 24
    target = torch.softmax(torch.randn(n, vocab, generator=torch.Generator().manual_seed(2)) * 2, 1)
    target[:, vocab - vocab // 6:] = 0
    target[:, vocab - 5] = 2.0 ** -100
    assert next_tokens(target, torch.ones(n)) == [vocab - 5] * n
    target[:, vocab // 3:] = 0
    target[:, vocab // 2] = 2.0 ** -149
    assert next_tokens(target, torch.full((n,), 2.0)) == [vocab // 2] * n
