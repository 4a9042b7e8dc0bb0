"""The attention over packed rows winds down when its waits run out.

A test-only fault makes the decoding warps withhold a tile's announcement, with a
short limit per wait: the wait of the second product's issuer runs out, then those
for that product (softmax, decoding) and for what the decoding no longer makes.  The
call returns with DSA_ERR_TIMEOUT at one of the kernel's wait sites and NaN in every
row that has keys, and the next call is correct.  With and without key splits; rows
of one block, where only the end of the row waits, to many.
"""
import numpy as np
import pytest

from tests.test_int4_mla_gpu import Case

pytestmark = pytest.mark.gpu
SITES = set(range(41, 61))


@pytest.fixture(scope="module")
def N():
    from long_context_sparse_04_b200 import build
    build.build()
    from long_context_sparse_04_b200 import _native
    return _native


@pytest.mark.parametrize("T,klens", [(2, [900, 70]), (21, [1, 64, 65, 300, 600]), (80, [600, 0, 64, 1, 300]), (200, [0, 64, 130, 513, 2048, 1])])
@pytest.mark.parametrize("H", [128, 40])
def test_a_wait_that_runs_out_ends_the_call(N, T, klens, H):
    import torch
    c = Case(N, [klens[t % len(klens)] for t in range(T)], H=H, topk=1024, seed=T).build()
    torch.cuda.synchronize()
    N.dsa_set_fault_injection(1 << 12, N.DSA_FAULT_MLA_INT4_VALUES)
    try:
        c.call()
        out, lse = c.result()
    finally:
        N.dsa_set_fault_injection(0, 0)
    code, site = c.status()
    assert code == N.DSA_ERR_TIMEOUT and site in SITES, (code, site)
    keys = c.klen > 0
    assert np.isnan(out[:T][keys]).all() and np.isnan(lse[:T][keys]).all()
    assert (out[:T][~keys] == 0).all() and np.isneginf(lse[:T][~keys]).all()
    assert (out[T] == 55).all() and (lse[T] == 55).all(), "a row behind the last is written"
    # nothing of it is left: the same call without the fault
    c.call().check(rows=sorted({0, 1, T // 2, T - 1}))
    assert c.status() == (0, -1)


def test_a_short_limit_alone_changes_nothing(N):
    """Waits that are met do not run out at the limit of the test above."""
    c = Case(N, [700, 3, 0, 2048] * 30, topk=1024, seed=5).build()
    N.dsa_set_fault_injection(1 << 12, 0)
    try:
        c.call().check(rows=[0, 1, 2, 3, 119])
    finally:
        N.dsa_set_fault_injection(0, 0)
    assert c.status() == (0, -1)
