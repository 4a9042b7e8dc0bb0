"""dsa_batch_plan against the sequential oracle: whole numbers, so every output
is equal."""
import numpy as np
import pytest

from oracle import dsa_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def N():
    from long_context_sparse_04_b200 import build
    build.build()
    from long_context_sparse_04_b200 import _native
    return _native


class Plan:
    """Device state of a planner: lengths, free list, block table (or seq_start)."""

    def __init__(self, N, lens, table, free, num_pages, page, max_tokens, seq_start=None, num_tokens=None,
                 in_place=False, release=True):
        import torch
        self.N, self.torch = N, torch
        i32 = lambda x: torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
        B = len(lens)
        self.B, self.M, self.page = B, max_tokens, page
        self.seq_len, self.n_new = i32(lens), i32(np.zeros(B))
        self.release = i32(np.zeros(B)) if release else None
        self.seq_len_out = self.seq_len if in_place else i32(np.full(B, -7))
        self.paged = table is not None
        self.table = i32(table) if self.paged else None
        self.start = None if seq_start is None else i32(seq_start)
        self.free = i32(list(free) + [-9] * (num_pages - len(free))) if self.paged else None
        self.free_count = i32([len(free)])
        self.free_count_out = self.free_count if in_place else i32([-7])
        # one guard row behind each output
        self.out = {k: torch.full((max_tokens + 1,), -55, dtype=torch.int32, device="cuda") for k in ("row_seq", "row_klen", "tok_pos")}
        self.out["slot"] = torch.full((max_tokens + 1,), -55, dtype=torch.int64, device="cuda")
        self.tok_start = i32(np.full(B + 2, -55))
        self.totals = i32(np.full(5, -55))
        p = lambda x: None if x is None else x.data_ptr()  # noqa: E731
        self.cache = N.dsa_cache(block_table=p(self.table), seq_start=p(self.start), page_size=page if self.paged else 0,
                                 max_pages_per_seq=self.table.shape[1] if self.paged else 0, num_seqs=B,
                                 num_tokens=num_pages * page if self.paged else num_tokens)
        self.plan = N.dsa_plan(
            seq_len=p(self.seq_len), n_new=p(self.n_new), release=p(self.release), seq_len_out=p(self.seq_len_out),
            free_count=p(self.free_count) if self.paged else None, free_count_out=p(self.free_count_out) if self.paged else None,
            free_pages=p(self.free), free_capacity=num_pages if self.paged else 0, max_tokens=max_tokens,
            tok_start=p(self.tok_start), totals=p(self.totals), **{k: p(v) for k, v in self.out.items()})
        self.nb = N.dsa_workspace_size(None, None, N.DSA_OP_BATCH_PLAN)
        self.ws = torch.zeros(self.nb, dtype=torch.uint8, device="cuda")

    @property
    def stream(self):
        return self.torch.cuda.current_stream().cuda_stream

    def run(self, n_new, release=None):
        self.n_new.copy_(self.torch.as_tensor(np.asarray(n_new, np.int32)))
        if release is not None:
            self.release.copy_(self.torch.as_tensor(np.asarray(release, np.int32)))
        self.N.dsa_batch_plan(self.cache, self.plan, self.ws.data_ptr(), self.nb, self.stream)

    def status(self):
        return self.N.dsa_read_device_status(self.ws.data_ptr(), self.stream)

    def check(self, want, free_before=None):
        n, M = len(want["rows"]), self.M
        h = {k: v.cpu().numpy() for k, v in self.out.items()}
        assert self.totals.tolist() == want["totals"] + [-55]
        assert self.tok_start.tolist() == want["start"] + [-55]
        assert self.seq_len_out.tolist() == want["seq_len"]
        seq = np.array([r[0] for r in want["rows"]], int)
        pos = np.array([r[1] for r in want["rows"]], int)
        np.testing.assert_array_equal(h["row_seq"][:n], seq)
        np.testing.assert_array_equal(h["tok_pos"][:n], pos)
        np.testing.assert_array_equal(h["row_klen"][:n], pos + 1)
        np.testing.assert_array_equal(h["slot"][:n], np.array([r[2] for r in want["rows"]], int))
        assert (h["row_seq"][n:M] == (seq[-1] if n else 0)).all()
        assert (h["tok_pos"][n:M] == -1).all() and (h["slot"][n:M] == -1).all() and (h["row_klen"][n:M] == 0).all()
        assert all(h[k][M] == -55 for k in h), "a row behind max_tokens is written"
        if self.paged:
            np.testing.assert_array_equal(self.table.cpu().numpy(), want["block_table"])
            left = int(self.free_count_out[0])
            free = self.free.cpu().numpy()
            assert free[:left].tolist() == want["free_list"]
            if free_before is not None:
                keep = max(left, len(free_before))
                assert (free[keep:] == -9).all()


def make_state(rng, B, P, W, spare, fill=0.5):
    lens = rng.integers(0, int(W * P * fill) + 1, B)
    held = -(-lens // P)
    pages = rng.permutation(int(held.sum()) + spare)
    table = np.full((B, W), -1)
    o = 0
    for b in range(B):
        table[b, : held[b]] = pages[o: o + held[b]]
        o += held[b]
    return lens, table, pages[o:].tolist(), len(pages)


@pytest.mark.parametrize("B,P,W,hi,spare,M", [
    (1, 64, 4, 1, 3, 1), (1, 1, 5, 3, 2, 9), (7, 16, 10, 40, 30, 100), (33, 48, 9, 5, 0, 64), (256, 64, 64, 2, 100, 300),
    (1023, 7, 20, 9, 900, 3000), (1024, 64, 8, 3, 50, 777), (1025, 64, 8, 30, 3000, 16384), (3000, 32, 40, 70, 9000, 100003),
    (16384, 64, 6, 2, 4000, 20000), (5, 64, 4000, 100000, 6000, 131072), (40, 16, 30, 20, 0, 0)])
def test_plan_matches_oracle(N, B, P, W, hi, spare, M):
    rng = np.random.default_rng(B * 1000 + hi)
    lens, table, free, num_pages = make_state(rng, B, P, W, spare)
    for with_release in (True, False):
        rel = (rng.random(B) < 0.15).astype(int) if with_release else None
        n_new = rng.integers(0, hi + 1, B)
        if with_release:
            n_new[rel > 0] = 0
        p = Plan(N, lens, table, free, num_pages, P, M, release=with_release)
        p.run(n_new, rel)
        want = R.batch_plan(lens, n_new, rel, free, table, P, num_pages, M)
        p.check(want, free)
        assert p.status() == ((0, -1) if want["error"][0] == "ok" else (N.DSA_ERR_OUT_OF_RANGE, want["error"][1]))
        assert N.dsa_read_kernel_trace(p.ws.data_ptr(), p.stream) == N.DSA_KERNEL_BATCH_PLAN


@pytest.mark.parametrize("M", [40, 5000])
def test_steps_in_place(N, M):
    """Lengths and free count updated in place over many steps, as a server runs
    it: requests grow, finish, hand their pages back and start again."""
    rng = np.random.default_rng(M)
    B, P, W = 61, 16, 12
    lens, table, free, num_pages = make_state(rng, B, P, W, 60, fill=0.3)
    p = Plan(N, lens, table, free, num_pages, P, M, in_place=True)
    for step in range(12):
        rel = (rng.random(B) < 0.2).astype(int)
        n_new = np.where(rel > 0, 0, rng.integers(0, 30, B))
        p.run(n_new, rel)
        want = R.batch_plan(lens, n_new, rel, free, table, P, num_pages, M)
        p.check(want)
        lens, table, free = want["seq_len"], want["block_table"], want["free_list"]
        p.status()


def test_contiguous(N):
    rng = np.random.default_rng(3)
    start = np.array([0, 100, 260, 300], int)
    lens = np.array([90, 0, 39, 50])
    for n_new, M in ([5, 7, 1, 50], 100), ([5, 7, 2, 51], 100), ([0, 0, 0, 0], 3), ([10, 160, 1, 1], 11):
        p = Plan(N, lens, None, [], 0, 1, M, seq_start=start, num_tokens=400)
        p.run(n_new)
        want = R.batch_plan(lens, n_new, None, [], None, 1, 0, M, seq_start=start, num_tokens=400)
        p.check(want)
        assert p.status() == ((0, -1) if want["error"][0] == "ok" else (N.DSA_ERR_OUT_OF_RANGE, want["error"][1]))
    p = Plan(N, [3], None, [], 0, 1, 8, num_tokens=10)           # one sequence from row 0, seq_start NULL
    p.run([7])
    p.check(R.batch_plan([3], [7], None, [], None, 1, 0, 8, num_tokens=10))


@pytest.mark.parametrize("kind", ["neg_len", "neg_new", "past_table", "release_and_new", "too_long", "bad_free", "bad_table",
                                  "two", "huge"])
def test_bad_requests(N, kind):
    """A request in error is refused and named; the others are planned."""
    rng = np.random.default_rng(11)
    B, P, W, M = 2100, 16, 8, 9000
    lens, table, free, num_pages = make_state(rng, B, P, W, 3000, fill=0.4)
    n_new, rel = rng.integers(0, 4, B), np.zeros(B, int)
    bad = 1501
    n_new[bad] = 2
    if kind == "neg_len":
        lens[bad] = -1
    elif kind == "neg_new":
        n_new[bad] = -2 ** 31
    elif kind == "past_table":
        lens[bad] = P * W + 1
    elif kind == "release_and_new":
        rel[bad] = 1
    elif kind == "too_long":
        n_new[bad] = P * W - lens[bad] + 1
    elif kind == "huge":
        n_new[bad] = 2 ** 31 - 1
    elif kind == "bad_free":
        free[-1 - 3] = num_pages
        free[-1 - 9] = -5
    elif kind == "bad_table":
        lens[bad] = P + 3
        table[bad, 1] = num_pages + 7
    else:
        lens[bad] = -1
        n_new[700] = P * W + 1
    p = Plan(N, lens, table, free, num_pages, P, M)
    p.run(n_new, rel)
    want = R.batch_plan(lens, n_new, rel, free, table, P, num_pages, M)
    p.check(want)
    code = {"invalid": N.DSA_ERR_INVALID_ARG, "range": N.DSA_ERR_OUT_OF_RANGE}[want["error"][0]]
    assert p.status() == (code, want["error"][1])
    assert want["error"][1] == (700 if kind == "two" else bad) or kind == "bad_free"


@pytest.mark.parametrize("count", [-1, 1 << 30])
def test_bad_free_count(N, count):
    lens, table, free, num_pages = make_state(np.random.default_rng(5), 9, 16, 8, 20)
    p = Plan(N, lens, table, free, num_pages, 16, 64)
    p.free_count.fill_(count)
    n_new = [1, 20, 0, 1, 3, 1, 40, 0, 2]
    p.run(n_new)
    want = R.batch_plan(lens, n_new, None, [], table, 16, num_pages, 64)
    p.check(want)
    assert p.status() == (N.DSA_ERR_INVALID_ARG, -1)


def test_capture_replay_and_second_stream(N):
    """A captured plan updated in place advances the state at every replay."""
    import torch
    rng = np.random.default_rng(8)
    B, P, W, M = 19, 16, 20, 19
    lens, table, free, num_pages = make_state(rng, B, P, W, 40, fill=0.3)
    p = Plan(N, lens, table, free, num_pages, P, M, in_place=True)
    side = torch.cuda.Stream()
    p.n_new.fill_(1)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            N.dsa_batch_plan(p.cache, p.plan, p.ws.data_ptr(), p.nb, torch.cuda.current_stream().cuda_stream)
        for _ in range(37):
            g.replay()
    side.synchronize()
    for _ in range(37):
        want = R.batch_plan(lens, [1] * B, None, free, table, P, num_pages, M)
        lens, table, free = want["seq_len"], want["block_table"], want["free_list"]
    p.check(want)
    assert p.status() == (0, -1)


def test_workspace_shared_with_other_calls(N):
    """Plans between appends, reads and attention on one workspace, all on one stream."""
    import torch
    rng = np.random.default_rng(8)
    lens, table, free, pages = make_state(rng, 6, 64, 20, 30)
    pl = Plan(N, lens, table, free, pages, 64, 3000, in_place=True)
    nb = 1 << 20
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    pl.ws, pl.nb = ws, nb
    d = N.dsa_dims(n_idx_heads=64, d_idx=128, n_heads=128, d_c=512, d_r=64, topk=64, idx_dtype=N.DSA_FP8_E4M3,
                   mla_dtype=N.DSA_INT4, sm_scale=0.05, algo=0)
    lat = torch.zeros((pages * 64, N.dsa_latent_row_bytes(d)), dtype=torch.uint8, device="cuda")
    ik, isc = torch.zeros((pages * 64, 128), dtype=torch.uint8, device="cuda"), torch.zeros(pages * 64, device="cuda")
    cache = N.dsa_cache(latent=lat.data_ptr(), idx_k=ik.data_ptr(), idx_k_scale=isc.data_ptr(), block_table=pl.table.data_ptr(),
                        page_size=64, max_pages_per_seq=table.shape[1], num_seqs=6, num_tokens=pages * 64)
    k = torch.ones((3000, 128), device="cuda")
    new = torch.ones((3000, 576), dtype=torch.bfloat16, device="cuda")
    back = torch.empty_like(new)
    cur = dict(seq_len=lens, block_table=table, free_list=free)
    for step in range(4):
        n_new = rng.integers(0, 40, 6)
        want = R.batch_plan(cur["seq_len"], n_new, None, cur["free_list"], cur["block_table"], 64, pages, 3000)
        pl.run(n_new)
        slot = pl.out["slot"].data_ptr()
        N.dsa_cache_append_slots(d, cache, 3000, slot, k.data_ptr(), new.data_ptr(), ws.data_ptr(), nb, pl.stream)
        back.fill_(7)
        N.dsa_cache_read(d, cache, 3000, slot, None, back.data_ptr(), ws.data_ptr(), nb, pl.stream)
        n = int(pl.totals[0])
        assert n == len(want["rows"]) > 0
        assert (back[:n, 512:] == 1).all() and (back[n:] == 7).all()
        assert pl.status() == (0, -1)
        cur = want
