"""The debug-bounds build's checks of attention behind shared prefixes (parts of chunks, CTAs of a block) never fire,
and its results are right.  In a child process, so that this one keeps the release library."""
from __future__ import annotations

import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_debug_bounds_checks_of_shared_prefixes_pass():
    r = subprocess.run([sys.executable, os.path.join(HERE, "_debug_bounds_shared_child.py")], capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0, r.stderr[-3000:]
    rows = [json.loads(line) for line in r.stdout.splitlines() if line.startswith("{")]
    assert len(rows) == 10, r.stdout
    assert all(row["error_word"] == 0 for row in rows), rows
