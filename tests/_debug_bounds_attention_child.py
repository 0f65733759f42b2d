"""Child process of tests/test_debug_bounds_attention.py: attention calls whose
blocks are split over CTAs, through the library built with -DNVFP4_DEBUG_BOUNDS.
Prints the device error word of each case."""
from __future__ import annotations

import json
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [os.path.dirname(HERE), HERE]

import nvfp4_weight_quantized_gemv_gb300 as nv  # noqa: E402

nv.LIB_PATH = nv.DEBUG_LIB_PATH
from nvfp4_weight_quantized_gemv_gb300 import buildlib  # noqa: E402

buildlib.build(debug_bounds=True)
buildlib.build_binding()
assert nv.lib()._name == nv.DEBUG_LIB_PATH
from test_attention_ops import Paged, attn64, close_bf16, randn  # noqa: E402

# (tokens, lengths, query heads a kv head, kv heads, head_dim): records a block and a CTA, whole short blocks, the kernel
# for prompts with rows once, twice and four times, sequences that bring none, blocks that begin in a CTA's last units
CASES = [([1], [20000], 8, 1, 128), ([2, 0, 1], [9000, 30, 4000], 6, 2, 256), ([1] * 90, [1 + 97 * (i % 23) for i in range(90)], 4, 2, 128),
         ([1] * 40, [200] * 40, 8, 4, 128), ([3], [20001], 8, 1, 128), ([5] * 9, list(range(5, 1805, 200)), 8, 2, 64),
         ([700], [1900], 3, 2, 128), ([33, 0, 100], [400, 70, 3000], 6, 1, 256), ([17] * 12, list(range(20, 1000, 83)), 2, 2, 128)]
for qs, kvs, g, hkv, d in CASES:
    p = Paged(sum(kvs) + d, qs, kvs, hkv, d, 32)
    q = (randn(p.g, sum(qs), g * hkv, d) * 1.5).bfloat16().cuda()
    y = nv.nvfp4_attn_paged(q, *p.args(), max(qs), max(kvs))
    word = nv.nvfp4_device_error()
    ref, size = attn64(p, q.cpu(), d ** -0.5)
    close_bf16(y, ref, 2.0 ** -8 * size)
    print(json.dumps({"case": [qs[:3], kvs[:3], g, hkv, d], "error_word": word}), flush=True)
