"""How long the chunks of sequences' own tokens are, as host code: no GPU."""
from __future__ import annotations

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_weight_quantized_gemv_gb300", "csrc")

CODE = r"""
#include <cstdio>
#include "attn_units.h"
using namespace nvfp4;
int main() {
    const int most = 1 << 30;  // tokens of the longest sequence
    if (shared_chunk(0.f) != kChunkUnit || shared_chunk(1e30f) != most) return puts("ends"), 1;
    for (double least = 0.25; least < 1e12; least *= 1.0173) {
        const int n = shared_chunk((float)least);
        const double want = least < most ? least : most;
        // (a step of fp32 below at most)
        if (n % kChunkUnit || n > most || n < want * (1 - 1.2e-7) || n > want * (1 + 1.2e-7) + kChunkUnit)
            return printf("%g %d\n", least, n), 1;
        // a chunk's end, and their number, in 32 bits
        if ((long long)(most - 1) + n > 0x7FFFFFFF) return printf("overflow %g\n", least), 1;
    }
    puts("ok");
}
"""


def test_chunks_are_as_long_as_wanted_up_to_the_longest_sequence(tmp_path):
    (tmp_path / "chunks.cpp").write_text(CODE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, str(tmp_path / "chunks.cpp"), "-o", str(tmp_path / "chunks")], check=True)
    assert subprocess.run([str(tmp_path / "chunks")], capture_output=True, text=True).stdout == "ok\n"
