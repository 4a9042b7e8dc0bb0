"""A serving loop over a cache with 4-bit latents: batch plan, append by slot,
then dsa_decode_step on the padded batch, step after step, against the oracle."""
import numpy as np
import pytest

from long_context_sparse_04_b200 import inputs as I
from oracle import dsa_ref as R
from tests import parity as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def N():
    from long_context_sparse_04_b200 import build
    build.build()
    from long_context_sparse_04_b200 import _native
    return _native


@pytest.mark.parametrize("int4", [True, False])
@pytest.mark.parametrize("captured", [False, True])
def test_serving_loop(N, captured, int4):
    import torch
    from long_context_sparse_04_b200.workload import DevicePlanner, PagedCache
    rng = np.random.default_rng(3)
    B, page, M, topk = 5, 64, 40, 128
    pl = DevicePlanner(num_seqs=B, page_size=page, num_pages=60, max_pages_per_seq=12, max_tokens=M)
    ca = PagedCache(pl, n_heads=128, topk=topk, int4=int4)
    logical = [dict(k=np.zeros((0, 128), np.float32), lat=np.zeros((0, 576), np.uint16)) for _ in range(B)]
    steps = [([30, 0, 5, 1, 4], None), ([1, 8, 1, 20, 1], None), ([0, 0, 0, 0, 0], [0, 0, 1, 0, 0]), ([9, 1, 28, 1, 1], None),
             ([1, 1, 1, 1, 1], None)]
    q_idx = torch.empty((M, 64, 128), dtype=torch.uint8, device="cuda")
    q_scale, w = torch.empty((M, 64), device="cuda"), torch.empty((M, 64), device="cuda")
    q = torch.empty((M, 128, 576), dtype=torch.bfloat16, device="cuda")
    k_new = torch.empty((M, 128), device="cuda")
    lat_new = torch.empty((M, 576), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((M, 128, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((M, 128), device="cuda")

    def step():
        pl.plan()
        ca.append(k_new, lat_new)
        ca.decode_step(q_idx, q_scale, w, q, out=out, lse=lse)

    graph = None
    for n, (n_new, rel) in enumerate(steps):
        pl.n_new.copy_(torch.tensor(n_new, dtype=torch.int32))
        pl.release.copy_(torch.tensor(rel or [0] * B, dtype=torch.int32))
        T = sum(n_new)
        k, lat = rng.standard_normal((M, 128)).astype(np.float32), rng.standard_normal((M, 576)).astype(np.float32)
        k[T:], lat[T:] = np.nan, np.nan                        # padding is data of no token
        qi, qs = I.to_e4m3_rows(rng.standard_normal((M, 64, 128)).astype(np.float32))
        wv = (rng.standard_normal((M, 64)) / 8).astype(np.float32)
        qv = I.to_bf16_bits((rng.standard_normal((M, 128, 576)) * 0.05).astype(np.float32))
        lat = I.to_bf16_bits(lat)
        for dst, src in ((q_idx, qi), (q_scale, qs), (w, wv), (k_new, k)):
            dst.copy_(torch.from_numpy(np.ascontiguousarray(src)))
        q.view(torch.int16).copy_(torch.from_numpy(qv.view(np.int16)))
        lat_new.view(torch.int16).copy_(torch.from_numpy(lat.view(np.int16)))
        out.fill_(9.0), lse.fill_(9.0)
        torch.cuda.synchronize()
        if not captured or n == 0:
            step()                                             # the first step runs eagerly: it warms the library up
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        torch.cuda.synchronize()
        assert pl.status() == (0, -1) and ca.status() == (0, -1)
        o = 0
        rows = []
        for b in range(B):
            if rel and rel[b]:
                logical[b] = dict(k=np.zeros((0, 128), np.float32), lat=np.zeros((0, 576), np.uint16))
            for _ in range(n_new[b]):
                logical[b]["k"] = np.concatenate([logical[b]["k"], k[o: o + 1]])
                logical[b]["lat"] = np.concatenate([logical[b]["lat"], lat[o: o + 1]])
                rows.append((b, len(logical[b]["k"])))
                o += 1
        assert pl.totals.tolist()[:3] == [T, pl.totals.tolist()[1], 0]
        assert pl.seq_len.tolist() == [len(x["k"]) for x in logical]
        go = out.double().cpu().numpy()
        gl = lse.double().cpu().numpy()
        gi = ca.indices().cpu().numpy()
        for t, (b, klen) in enumerate(rows):
            codes, s = R.quantise_keys(logical[b]["k"][:klen])
            kk = R.e4m3_decode(codes) * s.astype(np.float64)[:, None]
            sc = R.indexer_row(R.e4m3_decode(qi[t]) * qs[t].astype(np.float64)[:, None], wv[t].astype(np.float64), kk)
            sel = gi[t][gi[t] >= 0]
            assert len(sel) == min(topk, klen) and (np.diff(sel) > 0).all()
            own = R.topk_row(sc, topk)
            far = [x for x in set(sel) ^ set(own[own >= 0]) if abs(sc[x] - R.kth_score(sc, topk)) > 1e-3 * max(abs(R.kth_score(sc, topk)), P.rms(sc))]
            assert not far, f"step {n} row {t}: selection"
            kv = logical[b]["lat"][sel]
            kv = R.int4_unpack(R.int4_pack(kv, 512, 64), 512, 64) if int4 else R.bf16_decode(kv).astype(np.float64)
            ro, rl = R.sparse_mla_row(R.bf16_decode(qv[t]).astype(np.float64), kv, 512, ca.sm_scale)
            P.check_mla(go[t], gl[t], ro, rl, True, f"step {n} row {t}")
        assert (go[T:] == 0).all() and np.isneginf(gl[T:]).all()


@pytest.mark.parametrize("name", ["decode", "prefill"])
def test_workload_over_packed_rows(N, name):
    """dsa_decode_step and dsa_forward over the packed cache of a seeded workload."""
    import torch
    from long_context_sparse_04_b200.workload import DeviceWorkload
    cfg = (I.CONFIGS["decode_128k_paged"].replace(ctx_lo=1500, ctx_hi=5200, n_seqs=3) if name == "decode"
           else I.CONFIGS["prefill_8k"].replace(seq_len=700))
    inp = I.generate(cfg, threads=4)
    wl = DeviceWorkload(inp, int4=True)
    rows = R.int4_pack(inp["latent"], 512, 64)
    np.testing.assert_array_equal(wl.latent.cpu().numpy(), rows)
    if name == "decode":
        out, lse, scores, idx = wl.decode_step(debug=True)
        op = N.DSA_OP_DECODE_STEP
    else:
        out, lse, idx = wl.forward()
        op, scores = N.DSA_OP_FORWARD, None
    torch.cuda.synchronize()
    assert wl.status(op) == (0, -1)
    # the packed values are exact in bf16: the oracle runs on them as a bf16 cache
    plain = dict(inp, latent=I.to_bf16_bits(R.int4_unpack(rows, 512, 64).astype(np.float32)))
    pick = range(wl.T) if name == "decode" else [0, 1, 63, 64, 500, 699]
    P.check_rows(plain, pick, None if scores is None else P.to_np(scores), P.to_np(idx), P.to_np(out), P.to_np(lse))
