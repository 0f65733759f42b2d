"""Arithmetic of the pass over shared prefixes, as host code: no GPU."""
from __future__ import annotations

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_weight_quantized_gemv_gb300", "csrc")

CODE = r"""
#include <cstdio>
#include "attn_units.h"
using namespace nvfp4;
// Every unit lies in its owner's range, ranges follow each other, and no owner is beyond the last CTA.
bool shares(int U, int C, int step) {
    if (shared_begin(0, U, C) != 0 || shared_begin(C, U, C) != U) return false;
    for (int u = 0; u < U; u += u + step < U || u == U - 1 ? step : U - 1 - u) {
        const int c = shared_owner(u, U, C);
        if (c < 0 || c >= C || shared_begin(c, U, C) > u || shared_begin(c + 1, U, C) <= u) return false;
    }
    return true;
}
int main() {
    for (int U = 1; U < 700; ++U)
        for (int C = 1; C <= U && C <= kSharedMostCtas; ++C)
            if (!shares(U, C, 1)) return printf("%d %d\n", U, C), 1;
    for (int C = 1; C <= kSharedMostCtas; ++C)
        if (!shares(kSharedMostUnits - 1, C, 9973) || !shares(kSharedMostUnits - 1 - C, C, 65521)) return printf("%d\n", C), 1;
    for (int kv = 128; kv < 5000; kv += 128)  // a group's rows see all of its prefix, whatever their block
        for (int rb = 0; rb < 5; ++rb)
            if (prompt_block_tiles(3, 200, kv, rb, false) != kv / 128) return printf("tiles %d\n", kv), 1;
    puts("ok");
}
"""


def test_units_of_the_pass_over_prefixes_are_shared_without_gap(tmp_path):
    (tmp_path / "units.cpp").write_text(CODE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, str(tmp_path / "units.cpp"), "-o", str(tmp_path / "units")], check=True)
    assert subprocess.run([str(tmp_path / "units")], capture_output=True, text=True).stdout == "ok\n"
