"""Arithmetic and host code around the attention operators: no GPU."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_weight_quantized_gemv_gb300", "csrc")

UNITS = r"""
#include <cstdio>
#include <cstdlib>
#include "attn_units.h"
int main(int, char **a) {  // as a warp adds them up: 32-bit sums of the lanes' two summands
    unsigned low = 0, high = 0;
    for (int lane = 0; lane < 32; ++lane) {
        const long long n = nvfp4::prompt_units(atoi(a[1]), atoi(a[2]), atoi(a[3]), lane, 32);
        low += nvfp4::units_low(n);
        high += nvfp4::units_high(n);
    }
    printf("%lld\n", nvfp4::units_joined(low, high));
}
"""


@pytest.fixture(scope="module")
def units(tmp_path_factory):
    at = tmp_path_factory.mktemp("units")
    (at / "units.cpp").write_text(UNITS)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, str(at / "units.cpp"), "-o", str(at / "units")], check=True)
    return lambda *n: int(subprocess.run([str(at / "units")] + [str(i) for i in n], check=True, capture_output=True).stdout)


@pytest.mark.parametrize("g,q_len,kv_len", [
    (8, 3_000_000, 3_000_000), (16, 2_200_000, 2_200_000), (64, 1 << 20, 1 << 20), (64, 1 << 18, 1 << 23),
    (1, 1 << 30, 1 << 30), (1, 1, 1), (3, 129, 1000), (8, 7, 0), (5, 300, 20)])
def test_units_of_a_prompt_do_not_wrap(units, g, q_len, kv_len):
    rows, want = q_len * g, 0
    blocks = -(-rows // 128)
    for rb in range(blocks) if blocks < 10000 else ():
        last = (min((rb + 1) * 128, rows) - 1) // g
        want += max(1, -(-(kv_len - q_len + last + 1) // 128)) + 6
    got = units(g, q_len, kv_len)
    if blocks < 10000:
        assert got == want
    else:  # tiles of a block lie between those without rounding and one more
        most = blocks * (kv_len / 128 + 7) - (q_len / 128) * (blocks - 1) / 2
        assert most - 1.01 * blocks - 10 <= got <= most + 10


def test_the_library_is_built_without_pytorch():
    """-S: no site packages.  The library is there afterwards, and the binding is said not to be."""
    for code in ("-m", "nvfp4_weight_quantized_gemv_gb300.buildlib"), ("-c", "import nvfp4_weight_quantized_gemv_gb300 as nv; "
                                                                     "print(nv.build())"):
        r = subprocess.run([sys.executable, "-S", *code], cwd=ROOT, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        path = r.stdout.splitlines()[0]
        assert path.endswith("libnvfp4_gemv.so") and os.path.exists(path)
        assert "_attn_binding.so" not in r.stdout


def test_a_binding_for_another_pytorch_is_built_anew_and_not_loaded(monkeypatch):
    pytest.importorskip("torch")
    import nvfp4_weight_quantized_gemv_gb300 as nv
    from nvfp4_weight_quantized_gemv_gb300 import buildlib

    nv.build()
    assert buildlib.binding_made_for() == buildlib.binding_fits()
    made = os.path.getmtime(buildlib.build_binding())
    assert os.path.getmtime(buildlib.build_binding()) == made

    monkeypatch.setattr(nv, "_attn", None)
    nv._attn_setup()
    monkeypatch.setattr(nv, "_attn", None)
    with monkeypatch.context() as m:
        m.setattr(buildlib, "binding_fits", lambda: "another")
        with pytest.raises(RuntimeError, match="another Python or PyTorch"):
            nv._attn_setup()

    commands = []

    def run(cmd, **kw):  # no compiler: the command is what is looked at
        commands.append(cmd)
        return subprocess.CompletedProcess(cmd, 1, "", "not run")

    with monkeypatch.context() as m:
        m.setattr(buildlib, "binding_made_for", lambda: "another")
        m.setattr(buildlib.subprocess, "run", run)
        with pytest.raises(RuntimeError, match="not run"):
            buildlib.build_binding()
    assert len(commands) == 1 and buildlib.BINDING_SOURCE in commands[0]
    assert buildlib.binding_made_for() == buildlib.binding_fits()


@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("short", [0, 1, 13, 200])
def test_append_counts_its_pages_in_64_bits(page, short):
    """max_q_len within a page of 2^31: the pages that a sequence touches are 2^31 / page, with 80000 heads too many."""
    import nvfp4_weight_quantized_gemv_gb300 as nv

    nv.build()
    tokens = 2 ** 31 - 1 - short
    kv = nv.nvfp4_head_rows(4096, 16, 16, 40000)
    how = nv.nvfp4_norm_rope(None, None, 0.0, None, 0, 0, 0)
    cache = nv.nvfp4_kv_cache(4096, 4096, 4096, 4096, 40000 * 16 * page, 16 * page, 16, 8, 40000, page, 16)
    batch = nv.nvfp4_kv_batch(4096, 4096, 4096, 1, 8, tokens, tokens, 8 * page)
    status = nv.lib().nvfp4_kv_append(None, kv, kv, how, cache, batch, None, None)
    assert status == nv.NVFP4_ERR_INVALID_ARG and "too large" in nv.nvfp4_last_error()
