"""What the plan counts over the steps of a server (rows, pages taken, requests refused,
pages handed back), from the logical lengths alone."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,captured", [(16, False), (64, False), (64, True)])
def test_totals_follow_from_the_lengths(page, captured):
    import torch
    from long_context_sparse_04_b200.workload import DevicePlanner
    rng = np.random.default_rng(page)
    B, M, pages = 23, 400, 900
    pl = DevicePlanner(num_seqs=B, page_size=page, num_pages=pages, max_pages_per_seq=40, max_tokens=M)
    up = lambda n: -(-n // page)  # noqa: E731
    length = np.zeros(B, int)
    taken = back = 0
    graph = None
    for step in range(30):
        rel = (rng.random(B) < 0.15) & (length > 0)
        n_new = np.where(rel, 0, rng.integers(0, 17, B))
        n_new = np.where(length + n_new > 40 * page, 0, n_new)
        pl.n_new.copy_(torch.as_tensor(n_new.astype(np.int32)))
        pl.release.copy_(torch.as_tensor(rel.astype(np.int32)))
        if captured and step == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                pl.plan()
        graph.replay() if graph else pl.plan()
        new = np.where(rel, 0, length + n_new)
        want_taken = int((up(length + n_new) - up(length))[~rel].sum())
        want_back = int(up(length)[rel].sum())
        assert pl.totals.tolist() == [int(n_new.sum()), want_taken, 0, want_back], f"step {step}"
        length = new
        taken, back = taken + want_taken, back + want_back
        assert pl.seq_len.tolist() == length.tolist() and pl.status() == (0, -1)
        assert int(pl.free_count[0]) == pages - int(up(length).sum()) == pages - taken + back
    assert taken > 100 and back > 50
    held = np.concatenate([pl.block_table.cpu().numpy()[b, : up(length[b])] for b in range(B)])
    free = pl.free_pages.cpu().numpy()[: int(pl.free_count[0])]
    assert sorted(np.concatenate([held, free]).tolist()) == list(range(pages))
