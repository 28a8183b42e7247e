"""Calls of the 8-bit cache at the edges of what they accept, and the report of a wait that ran out."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import synth
from tests import test_kv8_gpu as base
from tests.test_kv8_gpu import DEV, ints, kv8  # noqa: F401  (the fixture)
from tests.test_kv8_model_gpu import SIMT1, TC1, i32, lib, make  # noqa: F401  (the fixture)

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


def test_one_row_of_any_stride(kv8):  # noqa: F811
    """With one row its stride means nothing, and torch gives such a dimension any."""
    g = torch.Generator(device=DEV).manual_seed(0)
    hq, hkv, D = 4, 2, 64
    wide = torch.randn(2, hq * D + 2 * hkv * D + 3, generator=g, device=DEV).bfloat16()
    q = wide[:, :hq * D].view(2, hq, D)[:1]
    k, v = (wide[:, (hq + i * hkv) * D:(hq + (i + 1) * hkv) * D].view(2, hkv, D)[:1] for i in (0, 1))
    out = torch.empty(2, hq * D + 3, dtype=torch.bfloat16, device=DEV)[:, :hq * D].view(2, hq, D)[:1]
    assert all(t.stride(0) % 4 == 3 for t in (q, k, v, out))
    pool, scales = kv8.new_cache(1, hkv, D)
    table, rs, kv = ints([[0]]), ints([0, 1]), ints([1])
    kv8.append(pool, scales, table, rs, kv, k, v)
    kv8.attention(q, pool, scales, table, rs, kv, out=out)
    want = v.repeat_interleave(hq // hkv, 1).float()
    assert ((out.float() - want).abs() <= 2.0 ** -3 * want.abs() + 2.0 ** -8).all()      # e4m3: half a step is 2^-4


@pytest.mark.parametrize("n", [3, 150])
def test_rows_of_nobody_and_rows_without_a_number(kv8, n):  # noqa: F811
    """Rows in front of the first sequence are zeros like those behind the last; a NaN or an infinity in a
    query makes its own rows NaN and no others."""
    rng = np.random.default_rng(n)
    hq, hkv, D = 8, 2, 64
    rs, kv, table, pool, scales = base.make_cache(rng, [(n, 333), (2, 40)], hkv, D)
    rs = rs + 2
    q = torch.from_numpy(rng.standard_normal((int(rs[-1]) + 2, hq, D))).to(torch.bfloat16)
    base.check_attention(kv8, q, pool, scales, table, rs, kv)
    pd, sd = torch.from_numpy(pool).to(DEV), torch.from_numpy(scales).to(DEV)
    args = (pd, sd, ints(table), ints(rs), ints(kv))
    lse = torch.empty(q.shape[:2], device=DEV)
    out = kv8.attention(q.to(DEV), *args, lse=lse)
    q[3, 5, 7], q[4, 1, 0], q[int(rs[1]), 0, 63] = float("nan"), float("inf"), float("-inf")
    lse2 = torch.empty(q.shape[:2], device=DEV)
    out2 = kv8.attention(q.to(DEV), *args, lse=lse2)
    bad = torch.isnan(q.float()).any(-1).to(DEV) | torch.isinf(q.float()).any(-1).to(DEV)
    assert int(bad.sum()) == 3
    assert torch.isnan(out2[bad]).all() and torch.isnan(lse2[bad]).all()
    assert torch.equal(out2[~bad], out[~bad]) and torch.equal(lse2[~bad], lse[~bad])


@pytest.mark.parametrize("shape", [SIMT1, TC1], ids=["simt", "tc"])
def test_a_wait_that_runs_out_in_a_context_with_the_cache(lib, shape):  # noqa: F811
    """The 8-bit attention's waits report to the word that sync reads, with and without tensor-core
    GEMMs: by the attention's own wait helper on a barrier that nothing completes."""
    from speculative_decoding_verify_token_gb300 import _lib
    w = synth.model_weights(shape, seed=0)
    m = make(lib, shape, w, max_batch=1, max_ctx=64, max_k=4)
    p = synth.prompt_tokens(1, 20, shape.vocab)
    m.prefill(0, i32(p[:-1]))
    m.verify([0], i32(p[-1:]), i32([[0] * 4]), torch.zeros(1, 5, device=DEV), 0.0)
    m.sync()                                     # nothing has run out
    for bad in (0, 2001):
        with pytest.raises(_lib.SpecError) as e:
            m.check_wait_timeout(bad)
        assert e.value.code == _lib.SPEC_E_INVAL
    m.check_wait_timeout(50)
    for _ in range(2):
        with pytest.raises(_lib.SpecError) as e:
            m.sync()
        assert e.value.code == _lib.SPEC_E_TIMEOUT
    m.close()
    m = make(lib, shape, w, max_batch=1, max_ctx=64, max_k=4)
    m.prefill(0, i32(p[:-1]))
    m.sync()
    m.close()
