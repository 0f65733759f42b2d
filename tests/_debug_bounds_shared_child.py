"""Child process of tests/test_debug_bounds_shared.py: attention behind shared prefixes through the library built
with -DNVFP4_DEBUG_BOUNDS.  Prints the device error word of each case."""
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
from test_attention_ops import attn64, close_bf16  # noqa: E402
from test_shared_prefix import CASES, Shared, queries  # noqa: E402

for qs, kvs, groups, prefixes, g, hkv, d, page in CASES[::3] + [([1] * 5, [9000 + i for i in range(5)], [0, 5], [8960], 6, 2, 256, 64)]:
    p = Shared(sum(kvs) + d, qs, kvs, groups, prefixes, hkv, d, page)
    q = queries(p, g)
    y = p.call(q)
    word = nv.nvfp4_device_error()
    ref, size = attn64(p, q.cpu(), d ** -0.5)
    close_bf16(y, ref, 2.0 ** -8 * size)
    print(json.dumps({"case": [qs[:3], kvs[:3], g, hkv, d], "error_word": word}), flush=True)
