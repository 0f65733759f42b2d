"""Attention whose work does not fill the GPU, with workspaces that hold anything before the call."""
from __future__ import annotations

import pytest
import torch

import nvfp4_weight_quantized_gemv_gb300 as nv
from test_attention_ops import Paged, built, check_attn, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("qs,kvs,g,d", [([20], [200], 4, 256), ([40, 9], [41, 130], 2, 128), ([1, 2], [100, 300], 4, 128),
                                        ([2, 1], [3000, 9], 8, 128), ([17], [17], 1, 128)])
@pytest.mark.parametrize("byte", [0x00, 0x7F, 0x80, 0xFF])
def test_few_units_and_any_workspace(qs, kvs, g, d, byte):
    p = Paged(sum(kvs) + d, qs, kvs, 1, d, 32)
    q = randn(p.g, sum(qs), g, d).bfloat16().cuda()
    ws = torch.full((nv.nvfp4_attn_workspace_size(),), byte, dtype=torch.uint8, device="cuda")
    assert torch.equal(check_attn(p, q, workspace=ws), nv.nvfp4_attn_paged(q, *p.args(), max(qs), max(kvs)))
