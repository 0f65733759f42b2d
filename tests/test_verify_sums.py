"""How exactly verification weighs: thresholds placed next to a cumulative sum of the definition.

One entry of a row is chosen so that the cumulative sum with it lies 2^-41 to 2^-39 of the total above or below u_next times
the total, all taken exactly (math.fsum).  The kernel's sums are off by some 2^-46 of the total (a lane's batch, of weights
of any size, by half a step of its second fp32 number, 2^-49, for each of its at most 32 entries with signs that mostly
cancel; ten additions of pairs behind them by 2^-47 each), so it has to see on which side of the threshold the sum lies.
Sums kept to 2^-38 or less of the total fail here.
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


def place(r, i, above):
    """(u, x, token): with r[i] = x the sum up to i lies next to u times the total, and the definition takes `token`."""
    before, behind = math.fsum(r[:i]), math.fsum(r[i + 1:])
    u = float(torch.tensor((before + 0.5 * r[i]) / (before + behind + r[i])).float())
    total = before + behind
    gap = 2.0 ** -40 * total * (1 if above else -1)
    x = float(torch.tensor((u * total - before + gap) / (1 - u), dtype=torch.float64).float())
    if x <= 0:
        return None
    # the sum's distance from the threshold, without rounding errors that matter: products by 1 - u and u in two parts
    total += x
    far = math.fsum([before * (1 - u), x * (1 - u), -u * behind]) / total
    if not 2.0 ** -41 <= (far if above else -far) <= 2.0 ** -39:
        return None
    return u, x, i if above else next(j for j in range(i + 1, len(r)) if r[j] > 0)


def rows(seed, vocab, count, near):
    """Rows of a target, and of a draft model that is near it (None: no drafts), each with one entry that is placed."""
    g = torch.Generator().manual_seed(seed)
    target, draft, pick, want = [], [], [], []
    while len(pick) < count:
        x = torch.randn(vocab, generator=g) * 2
        p = torch.softmax(x, 0)
        q = torch.softmax(x + near * torch.randn(vocab, generator=g), 0) if near else torch.zeros(vocab)
        r = (p.double() - q.double()).clamp(min=0)
        share = r / r.sum()
        fit = ((share > 2.0 ** -22) & (share < 2.0 ** -18)).nonzero()[:, 0]
        i = int(fit[torch.randint(len(fit), (1,), generator=g)])
        found = place(r.tolist(), i, len(pick) % 2 == 0)
        if found is None:
            continue
        p[i], q[i] = found[1], 0.0
        target.append(p)
        draft.append(q)
        pick.append(found[0])
        want.append(found[2])
    return torch.stack(target), torch.stack(draft) if near else None, torch.tensor(pick), want


@pytest.mark.parametrize("scale", [0, -12, -30, -60, 50])
@pytest.mark.parametrize("vocab", [8000, 30001, 131072])
def test_thresholds_next_to_a_sum_of_the_target(vocab, scale):
    """Distributions of any scale: they need not be normalised."""
    n = 12
    target, _, pick, want = rows(vocab, vocab, n, 0)
    got = nv.nvfp4_verify_drafts((target * 2.0 ** scale).cuda(), torch.zeros(n, dtype=torch.int32).cuda(),
                                 torch.arange(n + 1, dtype=torch.int32).cuda(), torch.zeros(n).cuda(), pick.cuda())
    assert got[2].tolist() == want


@pytest.mark.parametrize("scale", [0, -30])
@pytest.mark.parametrize("near", [0.5, 1e-2, 1e-4])
@pytest.mark.parametrize("vocab", [8000, 30001, 131072])
def test_thresholds_next_to_a_sum_of_the_residual(vocab, near, scale):
    """Draft models far from the target and very near it, whose residual is a small part of either."""
    n = 12
    target, draft, pick, want = rows(vocab + 1, vocab, n, near)
    ids = torch.zeros(2 * n, dtype=torch.int32)
    ids[1::2] = (draft > target).int().argmax(1)  # refused by u = 1
    both = [torch.stack([t, torch.zeros_like(t)], 1).flatten(0, 1) * 2.0 ** scale for t in (target, draft)]
    got = nv.nvfp4_verify_drafts(both[0].cuda(), ids.cuda(), torch.arange(0, 2 * n + 1, 2, dtype=torch.int32).cuda(),
                                 torch.ones(2 * n).cuda(), pick.cuda(), draft=both[1].cuda())
    assert got[1].tolist() == [0] * n and got[2].tolist() == want
