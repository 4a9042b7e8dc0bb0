"""PagedCache layers that share one workspace against layers with their own: the same
bits, eagerly and in a captured graph."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def step_inputs(torch, M, topk, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    f = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    return dict(q_idx=(f(M, 64, 128) * 4).to(torch.float8_e4m3fn).view(torch.uint8), q_scale=f(M, 64).abs() * 0.01, w=f(M, 64) / 8,
                q=(f(M, 128, 576) * 0.05).bfloat16(), k_new=f(M, 128), lat_new=f(M, 576).bfloat16())


@pytest.mark.parametrize("captured", [False, True])
def test_shared_and_own_workspaces_agree(captured):
    import torch
    from long_context_sparse_04_b200.workload import DevicePlanner, PagedCache
    B, M, topk = 5, 24, 128
    results = []
    for shared in (False, True):
        pl = DevicePlanner(num_seqs=B, page_size=64, num_pages=60, max_pages_per_seq=12, max_tokens=M)
        first = PagedCache(pl, topk=topk)
        layers = [first] + [PagedCache(pl, topk=topk, int4=i != 2, workspace_of=first if shared and i != 2 else None) for i in (1, 2, 3)]
        ins = [step_inputs(torch, M, topk, i) for i in range(4)]
        outs = [(torch.zeros((M, 128, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((M, 128), device="cuda")) for _ in layers]
        if shared:
            assert layers[1]._ws is layers[3]._ws is first._ws

        def step():
            pl.plan()
            for c, x, (o, l) in zip(layers, ins, outs):
                c.append(x["k_new"], x["lat_new"])
                c.decode_step(x["q_idx"], x["q_scale"], x["w"], x["q"], out=o, lse=l)

        pl.n_new.copy_(torch.tensor([9, 1, 3, 0, 4], dtype=torch.int32))
        step()
        if captured:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        for _ in range(20):
            pl.n_new.copy_(torch.tensor([2, 4, 5, 6, 7], dtype=torch.int32))
            graph.replay() if captured else step()
        torch.cuda.synchronize()
        assert pl.status() == (0, -1) and all(c.status() == (0, -1) for c in layers)
        results.append([(o.clone(), l.clone(), c.indices().clone()) for (o, l), c in zip(outs, layers)])
        assert pl.seq_len.tolist() == [49, 81, 103, 120, 144]
    for a, b in zip(*results):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        assert not np.isnan(a[0].float().cpu().numpy()).any() and a[0].abs().sum() > 0


def test_refusals():
    from long_context_sparse_04_b200.workload import DevicePlanner, PagedCache
    kw = dict(num_seqs=2, page_size=64, num_pages=8, max_pages_per_seq=4, max_tokens=4)
    pl, other = DevicePlanner(**kw), DevicePlanner(**kw)
    small = PagedCache(pl, topk=16)
    with pytest.raises(ValueError, match="another planner"):
        PagedCache(other, topk=16, workspace_of=small)
    for kw in (dict(topk=2048), dict(topk=8), dict(topk=16, int4=False), dict(topk=16, n_heads=64), dict(topk=16, sm_scale=1.0),
               dict(topk=16, q_group=2)):
        with pytest.raises(ValueError, match="other sizes"):
            PagedCache(pl, workspace_of=small, **kw)
    assert PagedCache(pl, topk=16, workspace_of=small)._ws is small._ws
