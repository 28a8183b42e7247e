"""Calls of the 8-bit cache at the edges of what they accept."""
import os
import subprocess
import sys

import pytest

from tests.test_kv8_gpu import kv8  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PLANS = """
import numpy as np
from speculative_decoding_verify_token_gb300 import kv8
from tests import kv8_reference as ref
from tests.test_kv8_gpu import run_plan
rng = np.random.default_rng(0)
for B in (3054, 3055, 3060, 3071, 3073, 8192):
    kv, new = rng.integers(0, 50, B), rng.integers(0, 4, B)
    held = -(-kv // 16)
    table = np.full((B, 5), -1)
    pages = rng.permutation(B * 5)
    at = 0
    for b in range(B):
        table[b, :held[b]] = pages[at:at + held[b]]
        at += held[b]
    args = (kv, new, held, pages[at:], len(pages) - at, table, int(new.sum()) + 3)
    for g, w in zip(run_plan(kv8, *args), ref.plan(*args)):
        np.testing.assert_array_equal(g, w)
    print("ok", B)
"""


def test_plan_sizes_ascending_in_a_new_process(kv8):  # noqa: F811
    """A kernel's shared memory limit is the process's: batches around 48 KB of it, none of them after a
    larger one."""
    r = subprocess.run([sys.executable, "-c", PLANS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr[-2000:]
