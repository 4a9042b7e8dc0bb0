"""Batch plans whose finished requests hand back many pages."""
import numpy as np
import pytest

from oracle import dsa_ref as R
from tests.test_batch_plan_gpu import Plan, make_state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def N():
    from long_context_sparse_04_b200 import build
    build.build()
    from long_context_sparse_04_b200 import _native
    return _native


@pytest.mark.parametrize("B,P,W,M", [(1, 1, 5000, 4), (3, 1, 40000, 9), (200, 1, 300, 200), (200, 16, 2000, 256), (512, 1, 170, 2048),
                                     (513, 2, 400, 600), (300, 1, 1000, 4000), (2000, 4, 60, 3000)])
def test_pages_of_long_requests(N, B, P, W, M):
    """Runs of one request's pages and runs that cross requests, short ones between long
    ones, in the small and the large form."""
    rng = np.random.default_rng(B + W)
    lens, table, free, num_pages = make_state(rng, B, P, W, 50, fill=1.0)
    short = rng.random(B) < 0.4                    # their pages stay out of the cache's books: only a few are held
    for b in np.flatnonzero(short):
        keep = int(rng.integers(0, 3))
        used = -(-lens[b] // P)
        table[b, min(keep, used):] = -1
        lens[b] = min(lens[b], keep * P)
    for part in (0.02, 0.5, 1.0):
        rel = (rng.random(B) < part).astype(int)
        rel[rng.integers(0, B)] = 1
        n_new = np.where(rel > 0, 0, rng.integers(0, 3, B))
        n_new = np.where(lens + n_new > P * W, 0, n_new)
        p = Plan(N, lens, table, free, num_pages, P, M)
        p.run(n_new, rel)
        want = R.batch_plan(lens, n_new, rel, free, table, P, num_pages, M)
        p.check(want, free)
        assert p.status() == (0, -1)


def test_time_goes_with_the_pages(N):
    """A decoding batch that hands back 160,000 pages: by one CTA, a page a thread at a
    time, that took 347 us."""
    import torch
    B, P, W = 200, 16, 8192
    held = np.full(B, 4000)
    table = np.full((B, W), -1)
    table[:, :4000] = np.random.default_rng(1).permutation(B * 4000 + 300)[: B * 4000].reshape(B, 4000)
    free = sorted(set(range(B * 4000 + 300)) - set(table[:, :4000].ravel().tolist()))
    rel = (np.arange(B) % 5 == 0).astype(int)
    p = Plan(N, held * P, table, free, B * 4000 + 300, P, 256)
    p.run(1 - rel, rel)
    assert p.totals.tolist()[:4] == [160, 160, 0, 160000]
    us = []
    for _ in range(15):
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda._sleep(200000)
        a.record()
        N.dsa_batch_plan(p.cache, p.plan, p.ws.data_ptr(), p.nb, p.stream)
        b.record()
        torch.cuda.synchronize()
        us.append(a.elapsed_time(b) * 1e3)
    assert p.status() == (0, -1)
    assert np.median(us) < 120, f"{np.median(us):.0f} us"
