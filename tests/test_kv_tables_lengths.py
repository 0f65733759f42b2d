"""Lengths up to the last that 32 bits hold, in rows of the block table with pages for more."""
from __future__ import annotations

import pytest
import torch

import nvfp4_weight_quantized_gemv_gb300 as nv

pytestmark = pytest.mark.gpu

PAGE, WIDTH, MOST = 256, (1 << 23) + 1, (1 << 31) - 1


@pytest.fixture(scope="module")
def table():
    nv.build()
    assert nv.nvfp4_device_error() == 0
    return torch.arange(WIDTH, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def step(table, kv, q, tokens):
    got = nv.nvfp4_kv_tables(table, ints([WIDTH]), ints([7] * 4), torch.tensor([0, 0]).cuda(), ints([kv]), ints([q]), PAGE, tokens,
                             kept=ints([WIDTH]))
    return nv.nvfp4_device_error(), [t.tolist() for t in got]


@pytest.mark.parametrize("q", [0, 1, 300, 5000])
def test_the_longest_sequence_is_served(table, q):
    kv = MOST - q
    error, (cu, lens, pos, slots, held, _) = step(table, kv, q, q + 2)
    assert error == 0 and cu == [0, q] and lens == [MOST] and held == [WIDTH]
    assert pos == list(range(kv, MOST)) + [0, 0]
    assert slots == [(WIDTH - 1 - p // PAGE) * PAGE + p % PAGE for p in range(kv, MOST)] + [-1, -1]


@pytest.mark.parametrize("kv,q", [(MOST, 1), (MOST - 4, 5), (MOST - 100, 357), (1 << 30, 1 << 30)])
@pytest.mark.parametrize("tokens", [10, 5000])
def test_one_token_more_is_refused(table, kv, q, tokens):
    error, (cu, lens, pos, slots, held, span) = step(table, kv, q, tokens)
    assert error == 256 and cu == [0, 0] and lens == [kv] and held == [WIDTH] and span == [0, 0]
    assert pos == [0] * tokens and slots == [-1] * tokens
