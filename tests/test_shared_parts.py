"""How much of a prefix a call shares: whole pages and multiples of 128 tokens that every token of the group sees.

What is shared is read through the table of the group's first sequence alone, so that the others' entries of it may be
any pages; what is not is read through each sequence's own.  Both are told from a page whose values are NaN, which makes
every row NaN that reads it, whatever its weight there: entries that are not read change no bit.
"""
from __future__ import annotations

import pytest
import torch

from test_attention_ops import built  # noqa: F401
from test_shared_prefix import Shared, check, ints, queries

pytestmark = pytest.mark.gpu

# (tokens and lengths of the sequences, groups, prefixes, kv heads, head_dim, page, arguments), tokens shared by each group
CASES = [
    (([1] * 4, [300, 310, 320, 330], [0, 4], [256], 1, 128, 16, {}), [256]),
    (([1] * 4, [300, 310, 320, 330], [0, 4], [255], 1, 128, 16, {}), [128]),
    (([1] * 4, [300, 310, 320, 330], [0, 4], [127], 1, 128, 16, {}), [0]),
    # as far as every token of the group sees, its own sequence's other new tokens among them
    (([1] * 3, [300, 129, 320], [0, 3], [256], 2, 128, 16, {}), [128]), (([1] * 3, [300, 128, 320], [0, 3], [256], 2, 128, 16, {}), [0]),
    (([5, 1], [133, 260], [0, 2], [128], 1, 256, 64, {}), [128]), (([6, 1], [133, 260], [0, 2], [128], 1, 256, 64, {}), [0]),
    (([30, 7], [800, 420], [0, 2], [640], 1, 256, 32, {}), [384]),
    # whole pages
    (([1] * 3, [900, 910, 920], [0, 3], [511], 1, 128, 256, {}), [256]), (([1] * 3, [900, 910, 920], [0, 3], [255], 1, 128, 256, {}), [0]),
    (([1] * 3, [900, 910, 920], [0, 3], [512], 1, 64, 256, {}), [512]),
    # a group's tokens up to their bound
    (([2] * 5, [520, 540, 513, 600, 700], [0, 5], [384], 1, 128, 64, {"max_group_tokens": 10}), [384]),
    (([2] * 5, [520, 540, 513, 600, 700], [0, 5], [384], 1, 128, 64, {"max_group_tokens": 9}), [0]),
    # sequences that bring or hold nothing count for nothing
    (([1, 0, 1, 1], [600, 0, 640, 610], [0, 4], [512], 1, 128, 64, {}), [512]), (([1, 1, 1], [600, 0, 640], [0, 3], [512], 2, 256, 64, {}), [512]),
    (([1, 0, 1], [600, 200, 640], [0, 3], [512], 1, 128, 64, {}), [512]), (([0, 1, 1], [600, 640, 700], [0, 3], [512], 1, 128, 64, {}), [512]),
    # several groups, one that may not be shared between them
    (([1] * 8, [700, 701, 702, 200, 129, 300, 900, 910], [0, 3, 6, 8], [640, 256, 768], 2, 128, 64, {}), [640, 128, 768]),
    (([1, 1, 30, 1, 1, 1], [700, 701, 702, 703, 720, 800], [0, 2, 3, 6], [640, 640, 512], 1, 128, 64, {}), [640, 0, 512]),
    (([1, 1, 8, 8, 1, 1], [700, 701, 702, 703, 720, 800], [0, 2, 4, 6], [640, 640, 512], 1, 128, 64, {"max_group_tokens": 15}), [640, 0, 512]),
    # more rows than a block, and more sequences than the plan keeps at hand
    (([1] * 40, [700 + i for i in range(40)], [0, 40], [640], 1, 128, 64, {}), [640]),
    (([1] * 1100, [160 + i % 50 for i in range(1100)], [0, 1100], [128], 1, 64, 16, {}), [128]),
]


@pytest.mark.parametrize("case,shared", CASES)
@pytest.mark.parametrize("g", [1, 4])
def test_what_is_read_once(case, shared, g):
    qs, kvs, groups, prefixes, hkv, d, page, kw = case
    p = Shared(sum(kvs) + g, qs, kvs, groups, prefixes, hkv, d, page)
    q = queries(p, g)
    y = check(p, q, **kw)
    if max(qs) * g >= 64:  # (they fill the tensor core's tiles by themselves)
        shared = [0] * len(shared)
    table = p.table.clone()
    nan = min(set(range(p.pages)) - set(table.flatten().tolist()))
    p.v.view(torch.uint8)[nan] = 0x7F

    def with_other_pages(where):  # the sequences that read any of these (sequence, column)
        t = table.clone()
        for b, c in where:
            t[b, c] = nan
        p.dev[0] = t.cuda()
        z = p.call(q, **kw)
        read = []
        for b in range(len(qs)):
            old, new = y[p.cu[b]:p.cu[b + 1]], z[p.cu[b]:p.cu[b + 1]]
            if torch.isnan(new).any():
                assert torch.isnan(new).all()
                read.append(b)
            else:
                assert torch.equal(new, old)
        return read

    for i, n in enumerate(shared):
        group = [b for b in range(groups[i], groups[i + 1]) if qs[b] > 0 and kvs[b] > 0]
        others = group[1:]
        if n > 0:
            assert with_other_pages([(b, c) for b in others for c in range(n // page)]) == []
            assert with_other_pages([(group[0], n // page - 1)]) == group
        reads = [b for b in others if kvs[b] > n]  # what is behind, each through its own row
        assert with_other_pages([(b, n // page) for b in reads]) == reads
        assert with_other_pages([(group[0], n // page)]) == (group[:1] if kvs[group[0]] > n else [])
    p.dev[0] = ints(table.tolist())
    assert torch.equal(p.call(q, **kw), y)
