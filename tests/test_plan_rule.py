"""The batch plan's admission, where one request holds up others (the oracle's rule, which
the kernel is compared with): no request overtakes one that waits."""
import numpy as np

from oracle import dsa_ref as R


def plan(n_new, max_tokens, free, lens=None, release=None):
    B = len(n_new)
    lens = [0] * B if lens is None else lens
    return R.batch_plan(lens, n_new, release, list(range(free)), np.full((B, 64), -1), 16, 64, max_tokens)


def test_a_request_of_too_many_rows_holds_up_those_behind_it():
    r = plan([3, 41, 1, 0, 2], 40, 20)
    assert r["start"] == [0, 3, 3, 3, 3, 3] and r["totals"] == [3, 1, 3, 0] and r["error"] == ("ok", -1)
    r = plan([3, 37, 1, 0, 2], 40, 20)                # as much as fits of it, and the rest waits for a step
    assert r["totals"] == [40, 4, 2, 0]


def test_a_request_that_waits_for_pages_holds_up_those_behind_it_that_need_some():
    r = plan([16, 33, 1, 5], 100, 3, lens=[0, 0, 0, 3])
    assert r["seq_len"] == [16, 0, 0, 8] and r["totals"][2] == 2


def test_requests_in_error_hold_up_no_one():
    r = plan([2, 16 * 64 + 1, -1, 2], 40, 20)
    assert r["totals"][:3] == [4, 2, 2] and r["error"] == ("range", 1)
