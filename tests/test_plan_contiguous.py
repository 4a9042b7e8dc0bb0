"""Batch plans of contiguous caches: a request gets rows of its own only.

The oracle is held to the property (CPU), the kernel to the oracle (GPU)."""
import numpy as np
import pytest

from oracle import dsa_ref as R


def layouts():
    """(name, seq_start or None, seq_len, n_new, num_tokens)"""
    yield "next_full", [0, 100, 260, 300], [90, 0, 39, 50], [5, 7, 2, 50], 400
    yield "next_exactly_full", [0, 100, 260, 300], [90, 0, 39, 50], [10, 160, 1, 50], 400
    yield "any_order", [300, 0, 260, 100], [50, 90, 39, 0], [51, 11, 2, 161], 400
    yield "any_order_fits", [300, 0, 260, 100], [50, 90, 39, 0], [50, 10, 1, 160], 400
    yield "idle_slots_at_row_0", [0, 0, 0, 128], [0, 60, 0, 9], [0, 3, 0, 2], 256
    yield "idle_next", [0, 100], [95, 0], [6, 0], 400
    yield "two_share_a_start", [0, 0, 128], [5, 7, 1], [1, 0, 1], 256
    yield "two_start_at_once", [64, 64, 128], [0, 0, 1], [4, 4, 1], 256
    yield "none_given", None, [3, 0, 0], [2, 0, 0], 10
    yield "none_given_two", None, [3, 0, 0], [2, 1, 0], 10
    yield "negative", [-4, 0], [1, 2], [1, 1], 64
    yield "beyond", [0, 500], [1, 0], [1, 1], 400
    yield "one", [7], [3], [12], 22
    yield "one_too_many", [7], [3], [13], 22
    rng = np.random.default_rng(5)
    for B in (2, 3, 255, 256, 257, 700):
        starts = np.cumsum(rng.integers(0, 40, B))
        room = np.append(starts[1:], starts[-1] + 20) - starts
        lens = (rng.random(B) * (room + 1)).astype(int)
        n_new = np.where(rng.random(B) < 0.7, rng.integers(0, 25, B), 0)
        perm = rng.permutation(B) if B % 2 else np.arange(B)
        yield f"random_{B}", starts[perm].tolist(), lens[perm].tolist(), n_new[perm].tolist(), int(starts[-1]) + 20


CASES = list(layouts())
IDS = [c[0] for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_slots_are_the_requests_own(case):
    _, start, lens, n_new, tokens = case
    B = len(lens)
    r = R.batch_plan(lens, n_new, None, [], None, 1, 0, 4096, seq_start=start, num_tokens=tokens)
    at = [0] * B if start is None else start
    held = {}                                    # row -> its request, before the step
    for b in range(B):
        for i in range(lens[b]):
            held.setdefault(at[b] + i, b)
    slots = [s for _, _, s in r["rows"]]
    assert len(set(slots)) == len(slots) and all(0 <= s < tokens for s in slots)
    for b, pos, s in r["rows"]:
        assert s == at[b] + pos
        assert s not in held, f"row {s} of request {held.get(s)} is given to request {b}"
        assert all(not at[b] < x <= s for x in at), f"row {s} lies behind another request's first"


def test_a_full_neighbour_refuses():
    r = R.batch_plan([90, 0, 39, 50], [5, 7, 2, 50], None, [], None, 1, 0, 100, seq_start=[0, 100, 260, 300], num_tokens=400)
    assert r["error"] == ("range", 2) and r["totals"] == [62, 0, 1, 0] and r["seq_len"] == [95, 7, 39, 100]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_plan_matches_oracle(case):
    from long_context_sparse_04_b200 import build
    build.build()
    from long_context_sparse_04_b200 import _native as N
    from tests.test_batch_plan_gpu import Plan
    _, start, lens, n_new, tokens = case
    for M in (4096, 61, 3000):
        for in_place in (False, True):
            p = Plan(N, lens, None, [], 0, 1, M, seq_start=start, num_tokens=tokens, in_place=in_place)
            p.plan.free_capacity = -5                # of the free list: not looked at
            p.run(n_new, [0] * len(lens))
            want = R.batch_plan(lens, n_new, None, [], None, 1, 0, M, seq_start=start, num_tokens=tokens)
            p.check(want)
            assert p.status() == ((0, -1) if want["error"][0] == "ok" else (N.DSA_ERR_OUT_OF_RANGE, want["error"][1]))


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1000, 16384])
def test_many_sequences_in_any_order(B):
    """The whole range of requests, half of them with full rows, in order and not."""
    from long_context_sparse_04_b200 import build
    build.build()
    from long_context_sparse_04_b200 import _native as N
    from tests.test_batch_plan_gpu import Plan
    rng = np.random.default_rng(B)
    room = rng.integers(1, 9, B)
    starts = np.cumsum(room) - room
    lens = (rng.random(B) * (room + 1)).astype(int)
    n_new = np.where(rng.random(B) < 0.5, room - lens, rng.integers(0, 4, B))
    tokens = int(room.sum())
    for perm in (np.arange(B), rng.permutation(B)):
        st, ln, nn, rm = starts[perm], lens[perm], n_new[perm], room[perm]
        p = Plan(N, ln, None, [], 0, 1, 8 * B, seq_start=st, num_tokens=tokens, release=False)
        p.run(nn)
        go = ln + nn <= rm
        got = np.where(go, nn, 0)
        n = int(got.sum())
        assert p.totals.tolist()[:4] == [n, 0, int((~go).sum()), 0]
        assert p.seq_len_out.tolist() == (ln + got).tolist()
        off = np.arange(n) - np.repeat(np.cumsum(got) - got, got)
        np.testing.assert_array_equal(p.out["slot"].cpu().numpy()[:n], np.repeat(st + ln, got) + off)
        assert p.status() == (N.DSA_ERR_OUT_OF_RANGE, int(np.flatnonzero(~go)[0]))
