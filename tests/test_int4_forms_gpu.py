"""Calls over packed rows that the documentation allows and the other tests leave out."""
import numpy as np
import pytest

from long_context_sparse_04_b200 import inputs as I
from oracle import dsa_ref as R
from tests.test_int4_mla_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def N():
    from long_context_sparse_04_b200 import build
    build.build()
    from long_context_sparse_04_b200 import _native
    return _native


@pytest.mark.parametrize("T", [3, 25, 60, 160])
def test_one_cache_from_row_0_for_every_sequence(N, T):
    """Neither a block table nor seq_start: row_seq plays no part, whatever it holds."""
    c = Case(N, [700 - 3 * t for t in range(T)], topk=300, seqs=[0] * T, page=0, seed=T).build()
    c.cache.seq_start = None
    c.d["seq"].copy_(c.torch.arange(T, dtype=c.torch.int32) * 1000 - 7)
    c.call().check(rows=[0, T // 2, T - 1])
    assert c.status() == (0, -1)


@pytest.mark.parametrize("T", [2, 30, 76])
def test_one_key_named_over_and_over(N, T):
    c = Case(N, [2048] * T, seqs=[0] * T, seed=T)
    c.idx[:] = 5
    c.idx[T - 1, ::2] = 2047
    c.build().call().check(rows=[0, T - 1])
    out, lse = c.result()
    one = R.int4_unpack(c.rows[c.physical(0, np.array([5]))], 512, 64)[0, :512]
    got = out[0]                                      # the mean of equal rows, rounded to bf16: weights of 1 and a sum of n
    assert (np.abs(got - one) <= 2.0 ** -8 * np.abs(one) + 2.0 ** -20).all()


@pytest.mark.parametrize("T", [4, 30, 90])
def test_lengths_change_between_replays(N, T):
    """A captured call over rows whose lengths and selections change in place, from nothing
    to everything and back."""
    import torch
    c = Case(N, [1500] * T, topk=1024, seqs=[0] * T, seed=T, poison=False).build()
    c.call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
    rng = np.random.default_rng(T)
    full = c.idx.copy()
    for kind in ("none", "one", "mixed", "full", "none"):
        n = {"none": np.zeros(T, int), "one": np.ones(T, int), "full": np.full(T, 1500)}.get(kind)
        n = rng.choice([0, 1, 64, 65, 300, 1500], T) if n is None else n
        c.klen = n.astype(np.int32)
        c.idx = np.full_like(full, -1)
        for t in range(T):
            k = min(1024, int(n[t]))
            c.idx[t, :k] = np.sort(rng.permutation(int(n[t]))[:k])
        c.d["klen"].copy_(torch.from_numpy(c.klen)), c.d["idx"].copy_(torch.from_numpy(c.idx))
        c.d["out"][:T] = 3.0
        g.replay()
        c.check(rows=sorted({0, 1, T // 2, T - 1}))
    assert c.status() == (0, -1)


@pytest.mark.parametrize("algo", ["STAGED", "SIMT"])
def test_decode_step_by_every_algorithm(N, algo):
    import torch
    from long_context_sparse_04_b200.workload import DeviceWorkload
    from tests import parity as P
    inp = I.generate(I.CONFIGS["decode_128k_paged"].replace(ctx_lo=900, ctx_hi=3100, n_seqs=2), threads=4)
    rows = R.int4_pack(inp["latent"], 512, 64)
    plain = dict(inp, latent=I.to_bf16_bits(R.int4_unpack(rows, 512, 64).astype(np.float32)))
    wl = DeviceWorkload(inp, int4=True, algo=getattr(N, "DSA_ALGO_" + algo))
    out, lse, scores, idx = wl.decode_step(debug=True)
    torch.cuda.synchronize()
    assert wl.status(N.DSA_OP_DECODE_STEP) == (0, -1)
    P.check_rows(plain, range(wl.T), P.to_np(scores), P.to_np(idx), P.to_np(out), P.to_np(lse))


def test_plans_on_two_streams_with_workspaces_of_their_own(N):
    import torch
    from tests.test_batch_plan_gpu import Plan, make_state
    made = []
    for B, P, W, M, seed in ((256, 16, 400, 256, 1), (1500, 64, 30, 9000, 2)):
        rng = np.random.default_rng(seed)
        lens, table, free, pages = make_state(rng, B, P, W, 2000)
        rel = (rng.random(B) < 0.3).astype(int)
        n_new = np.where(rel > 0, 0, rng.integers(0, 6, B))
        p = Plan(N, lens, table, free, pages, P, M)
        p.n_new.copy_(torch.as_tensor(n_new.astype(np.int32))), p.release.copy_(torch.as_tensor(rel.astype(np.int32)))
        made.append((p, R.batch_plan(lens, n_new, rel, free, table, P, pages, M), torch.cuda.Stream()))
    torch.cuda.synchronize()
    # (a plan that is not in place may run again: it writes what it wrote, except where pages
    # handed back have gone onto the list above the count it reads)
    for p, _, s in made:
        with torch.cuda.stream(s):
            N.dsa_batch_plan(p.cache, p.plan, p.ws.data_ptr(), p.nb, s.cuda_stream)
    for _ in range(20):
        for p, _, s in made:
            with torch.cuda.stream(s):
                N.dsa_batch_plan(p.cache, p.plan, p.ws.data_ptr(), p.nb, s.cuda_stream)
    torch.cuda.synchronize()
    for p, want, _ in made:
        p.check(want)
        assert p.status() == (0, -1)


def test_position_and_slot_write_the_same_bytes(N):
    """Appends by position into a cache with seq_start, and by the slots of a plan of it."""
    import torch
    d = N.dsa_dims(n_idx_heads=64, d_idx=128, n_heads=128, d_c=512, d_r=64, topk=64, idx_dtype=N.DSA_FP8_E4M3, mla_dtype=N.DSA_INT4,
                   sm_scale=0.05, algo=0)
    start, lens, n_new, tokens = [200, 0, 90], [3, 40, 0], [20, 50, 110], 300
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    st = torch.cuda.current_stream().cuda_stream
    from tests.test_batch_plan_gpu import Plan
    p = Plan(N, lens, None, [], 0, 1, 200, seq_start=start, num_tokens=tokens)
    p.run(n_new)
    assert p.totals.tolist()[:3] == [180, 0, 0]
    k, new = torch.randn(200, 128, device="cuda"), torch.randn(200, 576, device="cuda").bfloat16()
    got = []
    for by in ("slot", "position"):
        lat = torch.full((tokens, 416), 9, dtype=torch.uint8, device="cuda")
        ik, sc = torch.full((tokens, 128), 9, dtype=torch.uint8, device="cuda"), torch.full((tokens,), 9.0, device="cuda")
        s0 = i32(start)
        c = N.dsa_cache(latent=lat.data_ptr(), idx_k=ik.data_ptr(), idx_k_scale=sc.data_ptr(), seq_start=s0.data_ptr(), num_seqs=3,
                        num_tokens=tokens)
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        if by == "slot":
            N.dsa_cache_append_slots(d, c, 200, p.out["slot"].data_ptr(), k.data_ptr(), new.data_ptr(), ws.data_ptr(), 256, st)
        else:
            N.dsa_cache_append(d, c, 180, p.out["row_seq"].data_ptr(), p.out["tok_pos"].data_ptr(), k.data_ptr(), new.data_ptr(),
                               ws.data_ptr(), 256, st)
        assert N.dsa_read_device_status(ws.data_ptr(), st) == (0, -1)
        got.append((lat, ik, sc))
    assert all(torch.equal(a, b) for a, b in zip(*got)) and (got[0][2] != 9).sum() == 180
