"""Sparse MLA over packed 4-bit latent rows against float64 on the decoded rows.

Tolerances, from the arithmetic (u = 2^-8, half a bf16 step; e = 2^-24, half an
fp32 step; n keys, D dims):
  * the decoded rows are exact, products of bf16 are exact in fp32, a logit is a
    fp32 sum: |dz| <= Z with Z = 2 D e max_s sm_scale sum_d |q_d kv_sd| plus one
    rounding of sm_scale log2(e) and of the product, 4 e max|z|;
  * lse: dz, the exponential's 2^-22 and a sum of n positive terms:
        |dlse| <= Z + 2^-22 + n e + 4 e |lse|
  * out: each weight rounded to bf16 once (tensor cores; not CUDA cores), the
    logit's and the sum's errors, and the result rounded to bf16 once: with
    A = sum_s p_s |c_s|,
        |dout| <= (u + 2 (Z + 2^-22 + n e)) A + u |out| (1 + u) + 2^-126 (1 + sum_s |c_s|)
    the last term for underflow: a weight below 2^-126 of the largest may be
    flushed to zero, and so may a result below 2^-126 (bf16 and fp32 have the same
    smallest normal; q_std = 8 gives results of 1e-45).
"""
import numpy as np
import pytest

from long_context_sparse_04_b200 import inputs as I
from oracle import dsa_ref as R

pytestmark = pytest.mark.gpu
U, E = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module")
def N():
    from long_context_sparse_04_b200 import build
    build.build()
    from long_context_sparse_04_b200 import _native
    return _native


class Case:
    """Sequences of `ctx` tokens with packed rows, query rows of `klens`."""

    def __init__(self, N, klens, H=128, topk=2048, d_c=512, d_r=64, page=64, algo=0, q_std=0.05, seed=0, ctx=None,
                 spread=1.0, poison=True, seqs=None):
        import torch
        self.N, self.torch, self.algo = N, torch, algo
        rng = np.random.default_rng(seed)
        self.rng = rng
        self.T, self.H, self.topk, self.d_c, self.d_r = len(klens), H, topk, d_c, d_r
        self.klen = np.array(klens, np.int32)
        self.seq = np.arange(self.T, dtype=np.int32) if seqs is None else np.array(seqs, np.int32)
        B = int(self.seq.max()) + 1
        need = np.zeros(B, int)
        np.maximum.at(need, self.seq, np.maximum(self.klen, 1))
        if ctx is not None:
            need[:] = ctx
        unit = page or 64
        held = -(-need // unit)
        self.tokens = int(held.sum()) * unit
        lat = rng.standard_normal((self.tokens, d_c + d_r)) * np.exp(rng.uniform(-spread, spread, (self.tokens, 1)))
        self.rows = R.int4_pack(I.to_bf16_bits(lat.astype(np.float32)), d_c, d_r)
        starts = np.cumsum(held) - held
        self.page = page
        if page:
            perm = rng.permutation(int(held.sum()))
            self.table = np.full((B, int(held.max()) + 1), -1, np.int32)
            for b in range(B):
                self.table[b, : held[b]] = perm[starts[b]: starts[b] + held[b]]
        else:
            self.start = (starts * unit).astype(np.int32)
        self.idx = np.full((self.T, topk), -1, np.int32)
        for t in range(self.T):
            k = min(topk, int(self.klen[t]))
            self.idx[t, :k] = np.sort(rng.permutation(int(self.klen[t]))[:k])
        self.q = I.to_bf16_bits((rng.standard_normal((self.T, H, d_c + d_r)) * q_std).astype(np.float32))
        self.sm = np.float32(1 / np.sqrt(d_c + d_r))
        self.poison = poison

    def physical(self, t, sel):
        b = int(self.seq[t])
        if self.page:
            return self.table[b, sel // self.page].astype(np.int64) * self.page + sel % self.page
        return int(self.start[b]) + sel

    def selected(self, t):
        s = self.idx[t, : min(self.topk, int(self.klen[t]))].astype(np.int64)
        return s[s >= 0]

    def build(self):
        """Device copies; rows that no query selects hold NaN and wild bytes."""
        torch, N = self.torch, self.N
        rows = self.rows.copy()
        if self.poison:
            used = np.zeros(self.tokens, bool)
            for t in range(self.T):
                used[self.physical(t, self.selected(t))] = True
            rows[~used] = 0xFF
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        self.d = dict(rows=dev(rows), idx=dev(self.idx), seq=dev(self.seq), klen=dev(self.klen), q=dev(self.q.view(np.int16)),
                      out=torch.full((self.T + 1, self.H, self.d_c), 55.0, dtype=torch.bfloat16, device="cuda"),
                      lse=torch.full((self.T + 1, self.H), 55.0, device="cuda"))
        p = {k: v.data_ptr() for k, v in self.d.items()}
        self.dims = N.dsa_dims(n_idx_heads=64, d_idx=128, n_heads=self.H, d_c=self.d_c, d_r=self.d_r, topk=self.topk,
                               idx_dtype=N.DSA_FP8_E4M3, mla_dtype=N.DSA_INT4, sm_scale=float(self.sm), algo=self.algo)
        if self.page:
            self.d["table"] = dev(self.table)
            kw = dict(block_table=self.d["table"].data_ptr(), page_size=self.page, max_pages_per_seq=self.table.shape[1])
        else:
            self.d["start"] = dev(self.start)
            kw = dict(seq_start=self.d["start"].data_ptr())
        self.cache = N.dsa_cache(latent=p["rows"], num_seqs=int(self.seq.max()) + 1, num_tokens=self.tokens, **kw)
        self.r = N.dsa_rows(num_rows=self.T, row_seq=p["seq"], row_klen=p["klen"], max_klen=int(self.klen.max()), q_group=1)
        self.nb = N.dsa_workspace_size(self.dims, self.r, N.DSA_OP_SPARSE_MLA)
        self.ws = torch.zeros(self.nb, dtype=torch.uint8, device="cuda")
        return self

    @property
    def stream(self):
        return self.torch.cuda.current_stream().cuda_stream

    def call(self):
        p = {k: v.data_ptr() for k, v in self.d.items()}
        self.N.dsa_sparse_mla_fwd(self.dims, self.r, self.cache, p["q"], p["idx"], p["out"], p["lse"], self.ws.data_ptr(),
                                  self.nb, self.stream)
        return self

    def result(self):
        self.torch.cuda.synchronize()
        return self.d["out"].double().cpu().numpy(), self.d["lse"].double().cpu().numpy()

    def status(self):
        return self.N.dsa_read_device_status(self.ws.data_ptr(), self.stream)

    def ran(self):
        return self.N.dsa_read_kernel_trace(self.ws.data_ptr(), self.stream)

    def check(self, rows=None, skip=()):
        out, lse = self.result()
        assert (out[self.T] == 55).all() and (lse[self.T] == 55).all(), "a row behind the last is written"
        sm, tc = float(self.sm), self.algo != self.N.DSA_ALGO_SIMT
        for t in range(self.T) if rows is None else rows:
            sel = self.selected(t)
            sel = sel[~np.isin(sel, list(skip))]
            kv = R.int4_unpack(self.rows[self.physical(t, sel)], self.d_c, self.d_r)
            q = R.bf16_decode(self.q[t]).astype(np.float64)
            ro, rl = R.sparse_mla_row(q, kv, self.d_c, sm)
            if len(sel) == 0:
                assert (out[t] == 0).all() and np.isneginf(lse[t]).all(), f"row {t} selects nothing"
                continue
            n, D = len(sel), self.d_c + self.d_r
            z = sm * (q @ kv.T)
            Z = (2 * D * E * sm * (np.abs(q) @ np.abs(kv).T).max(1) + 4 * E * np.abs(z).max(1))
            ltol = Z + 2.0 ** -22 + n * E + 4 * E * np.abs(rl)
            assert (np.abs(lse[t] - rl) <= ltol).all(), f"row {t}: lse off by {np.abs(lse[t] - rl).max():.3e}, {ltol.max():.1e} allowed"
            p = np.exp(z - rl[:, None])
            A = p @ np.abs(kv[:, : self.d_c])
            w = (U if tc else 0.0) + 2 * (Z + 2.0 ** -22 + n * E)
            tol = w[:, None] * A + U * np.abs(ro) * (1 + U) + 2.0 ** -126 * (1 + np.abs(kv[:, : self.d_c]).sum(0))
            bad = np.abs(out[t] - ro) > tol
            assert not bad.any(), f"row {t}: {bad.sum()} of {bad.size} outputs outside; worst {np.abs(out[t] - ro).max():.3e}"


def algos(N):
    return {"auto": N.DSA_ALGO_AUTO, "simt": N.DSA_ALGO_SIMT}


SMALL = [0, 1, 2, 15, 16, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200]


@pytest.mark.parametrize("algo", ["simt", "auto"])
@pytest.mark.parametrize("page", [64, 0, 128, 192])
def test_short_rows(N, algo, page):
    c = Case(N, SMALL, page=page, algo=algos(N)[algo], seed=page).build().call()
    c.check()
    assert c.status() == (0, -1)


@pytest.mark.parametrize("T", [1, 2, 9, 18, 37, 74, 75])
def test_rows_and_splits(N, T):
    """From one row over every split count to one split a row."""
    rng = np.random.default_rng(T)
    k = [int(x) for x in rng.integers(1, 2500, T)]
    k[0] = 2300
    c = Case(N, k, seed=T).build().call()
    c.check(rows=sorted({0, T // 2, T - 1}))
    assert c.status() == (0, -1)
    first = [x.copy() for x in c.result()]
    again = c.call().result()
    for x, y in zip(first, again):
        np.testing.assert_array_equal(x, y)


@pytest.mark.parametrize("H", [8, 16, 24, 64, 72, 128])
@pytest.mark.parametrize("algo", ["simt", "auto"])
def test_heads(N, H, algo):
    c = Case(N, [70, 0, 333, 1], H=H, topk=300, algo=algos(N)[algo], seed=H).build().call()
    c.check()


@pytest.mark.parametrize("topk", [1, 7, 64, 100, 1000, 2047])
def test_topk_sizes(N, topk):
    c = Case(N, [1, topk, topk + 1, 2500, 0, 64], topk=topk, seed=topk).build().call()
    c.check()


@pytest.mark.parametrize("d_c,d_r,H", [(64, 16, 8), (32, 0, 16), (256, 64, 24), (512, 0, 8), (96, 8, 128)])
def test_other_dims_run_on_cuda_cores(N, d_c, d_r, H):
    c = Case(N, [0, 1, 40, 129], H=H, topk=100, d_c=d_c, d_r=d_r, seed=d_c, q_std=0.3).build().call()
    c.algo = N.DSA_ALGO_SIMT
    c.check()


def test_holes_repeats_and_any_order(N):
    """-1 within the selection, a key named twice, positions out of order."""
    c = Case(N, [900, 640, 64, 130], topk=640, seed=4)
    rng = np.random.default_rng(1)
    for t in range(c.T):
        k = min(c.topk, int(c.klen[t]))
        c.idx[t, :k] = rng.permutation(c.idx[t, :k])
        c.idx[t, rng.permutation(k)[: k // 3]] = -1
        c.idx[t, :2] = c.idx[t, 5]
    c.idx[2, :64] = -1                         # a whole block of holes, nothing left
    c.idx[1, 64:256] = -1                      # whole blocks of holes between keys
    c.idx[0, :128] = -1                        # holes first
    c.build().call().check()


@pytest.mark.parametrize("q_std", [1.0, 8.0, 60.0])
def test_large_logits(N, q_std):
    """Logits that grow along the row: the running maximum moves many times."""
    c = Case(N, [2048, 700, 129], seed=int(q_std), q_std=q_std, spread=2.0)
    c.build().call().check()


def test_extreme_rows(N):
    """Scales from subnormal to the largest, zero rows, a zero query."""
    c = Case(N, [256, 300], seed=3)
    c.rows[::7, 384:416] = 0x00
    c.rows[1::7, 384:416] = 0x03
    c.rows[2::7, 384:416] = 0x08
    c.rows[3::7, :256] = 0x88                  # code -8, which the writers never use
    c.q[1, 3] = 0
    c.build().call().check()


def test_bad_pages_are_skipped_and_named(N):
    c = Case(N, [200, 400, 64], seed=6)
    c.build()
    table = c.table.copy()
    table[1, 2] = c.tokens // c.page           # beyond the cache
    c.d["table"].copy_(c.torch.from_numpy(table))
    c.call()
    out, lse = c.result()
    assert c.status() == (N.DSA_ERR_OUT_OF_RANGE, c.tokens // c.page)
    c.check(rows=[0, 2])
    c.check(rows=[1], skip=range(128, 192))


def test_row_of_no_sequence(N):
    """A row_seq outside the cache reads nothing: zeros and -inf, named."""
    c = Case(N, [70, 80, 90], seed=7).build()
    c.d["seq"].copy_(c.torch.tensor([0, 3, 2], dtype=c.torch.int32))
    c.call()
    out, lse = c.result()
    assert (out[1] == 0).all() and np.isneginf(lse[1]).all()
    assert c.status()[0] == N.DSA_ERR_OUT_OF_RANGE
    c.check(rows=[0, 2])


def test_far_rows_pass_32_bits(N):
    """Byte offsets beyond 2^32 within the cache."""
    import torch
    c = Case(N, [640, 64], seed=8, page=64)
    big = (1 << 32) // 416 + 200000
    big += -big % 64
    shift = big // 64
    c.build()
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 5 GB")
    cache = torch.zeros((big + c.tokens, 416), dtype=torch.uint8, device="cuda")
    cache[big:] = c.d["rows"]
    c.d["rows"] = cache
    c.d["table"] += shift
    c.cache.latent, c.cache.num_tokens = cache.data_ptr(), big + c.tokens
    c.call().check()
    assert c.status() == (0, -1)


def test_noalloc_lse_null_and_prefill(N):
    """The call without a workspace gives the same bits; lse may be NULL; a prefill
    chunk of one sequence (more rows than one wave of clusters)."""
    T = 90
    c = Case(N, [500 + i for i in range(T)], topk=256, seqs=[0] * T, seed=9).build().call()
    c.check(rows=[0, 44, 89])
    out, lse = (x.copy() for x in c.result())
    p = {k: v.data_ptr() for k, v in c.d.items()}
    c.d["out"].fill_(55.0)
    N.dsa_sparse_mla_fwd_noalloc(c.dims, c.r, c.cache, p["q"], p["idx"], p["out"], None, c.stream)
    np.testing.assert_array_equal(c.result()[0], out)
    few = N.dsa_rows(num_rows=9, row_seq=p["seq"], row_klen=p["klen"], max_klen=600, q_group=1)
    c.d["out"][:9].fill_(55.0)
    N.dsa_sparse_mla_fwd_noalloc(c.dims, few, c.cache, p["q"], p["idx"], p["out"], p["lse"], c.stream)
    c.check(rows=[0, 4, 8])


def test_capture_replay_and_two_graphs(N):
    """Two captured calls that share a workspace, replayed one after the other with
    other inputs in place."""
    import torch
    a = Case(N, [300, 0, 2100, 64, 1], seed=10).build()
    b = Case(N, [1000, 129], seed=11).build()
    nb = max(a.nb, b.nb)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    a.ws = b.ws = ws
    a.nb = b.nb = nb
    a.call(), b.call()                          # warm
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            c.call()
        graphs.append(g)
    for c in (a, b):
        c.q = I.to_bf16_bits((np.random.default_rng(c.T).standard_normal(c.q.shape) * 0.2).astype(np.float32))
        c.d["q"].copy_(torch.from_numpy(c.q.view(np.int16)))
        c.d["out"][: c.T] = 1.0
    for _ in range(3):
        graphs[0].replay(), graphs[1].replay()
    a.check(), b.check()
    assert a.status() == (0, -1)


@pytest.mark.parametrize("kw,tc", [(dict(H=128), True), (dict(H=16), True), (dict(H=136), False), (dict(H=8, d_c=64, d_r=16), False),
                                   (dict(H=128, algo=1), False)])
def test_which_kernel_runs(N, kw, tc):
    """The tensor-core kernel takes every row of up to 128 heads of 512 + 64 dims."""
    c = Case(N, [70, 3], topk=100, seed=12, **kw).build().call()
    c.algo = N.DSA_ALGO_AUTO if tc else N.DSA_ALGO_SIMT
    c.check()
    assert c.ran() & (N.DSA_KERNEL_MLA_SIMT | N.DSA_KERNEL_MLA_INT4_TC) == (N.DSA_KERNEL_MLA_INT4_TC if tc else N.DSA_KERNEL_MLA_SIMT)


@pytest.mark.parametrize("seed", range(4))
def test_many_rows_of_every_length(N, seed):
    """More rows than pairs of SMs, in any order of lengths: a pair's blocks run on
    from row to row, over empty rows and rows of one block, odd and even."""
    rng = np.random.default_rng(seed)
    T = [77, 150, 223, 300][seed]
    k = rng.choice([0, 0, 1, 63, 64, 65, 128, 129, 192, 200, 256, 320, 500], T)
    if seed == 2:
        k[80:] = 0                                # whole pairs end in empty rows
    if seed == 3:
        k[:76] = 0                                # and begin with them
    k[5] = 300
    c = Case(N, [int(x) for x in k], topk=512, seed=seed, seqs=[int(x) for x in rng.integers(0, 9, T)]).build().call()
    c.check(rows=[int(x) for x in np.concatenate([np.arange(0, T, 7), np.flatnonzero(k == 1)[:5], [T - 1]])])
    assert c.status() == (0, -1)
    first = [x.copy() for x in c.result()]
    for x, y in zip(first, c.call().result()):
        np.testing.assert_array_equal(x, y)


@pytest.mark.parametrize("H", [1, 5, 63, 65, 127])
@pytest.mark.parametrize("T", [2, 21, 80])
def test_any_number_of_heads(N, H, T):
    """Rows merged from four, two and no key splits, heads that are no multiple of 8."""
    c = Case(N, [200 + 7 * t for t in range(T)], H=H, topk=300, seed=H + T).build().call()
    assert c.ran() & N.DSA_KERNEL_MLA_INT4_TC and c.status() == (0, -1)
    c.check(rows=sorted({0, 1, T // 2, T - 1}))


@pytest.mark.parametrize("T", [2, 21, 80])
def test_nan_and_infinite_queries_stay_with_their_head(N, T):
    c = Case(N, [500 + t for t in range(T)], topk=256, seed=T)
    c.q[0, 3, 5], c.q[1, 70, 575], c.q[T - 1, 127, 0] = 0x7FC0, 0x7F80, 0xFF80
    bad = [(0, 3), (1, 70), (T - 1, 127)]
    c.build().call()
    out, lse = c.result()
    assert c.status() == (0, -1)
    for t, h in bad:
        assert np.isnan(out[t, h]).all() and np.isnan(lse[t, h]), (t, h)
    keep = np.ones((T, 128), bool)
    keep[tuple(np.array(bad).T)] = False
    assert np.isfinite(out[:T][keep]).all() and np.isfinite(lse[:T][keep]).all()
    clean = Case(N, [500 + t for t in range(T)], topk=256, seed=T).build().call()
    o2, l2 = clean.result()
    np.testing.assert_array_equal(out[:T][keep], o2[:T][keep])
    np.testing.assert_array_equal(lse[:T][keep], l2[:T][keep])
    clean.check(rows=[0, T - 1])


def test_two_streams_at_once(N):
    """Two calls in flight on two streams, each with a workspace of its own."""
    import torch
    a = Case(N, [1500 + 3 * t for t in range(40)], topk=1024, seed=1).build()
    b = Case(N, [900 + 5 * t for t in range(9)], H=40, topk=512, seed=2).build()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        with torch.cuda.stream(s1):
            a.call()
        with torch.cuda.stream(s2):
            b.call()
    torch.cuda.synchronize()
    a.check(rows=[0, 39]), b.check(rows=[0, 8])
    assert a.status() == b.status() == (0, -1)


FIRST = """
import sys
sys.path.insert(0, {root!r})
import torch
from tests.test_int4_mla_gpu import Case
from long_context_sparse_04_b200 import _native as N
c = Case(N, [700] * {T}, topk=512).build()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    c.call()
for _ in range(2):
    g.replay()
c.check(rows=[0, {T} - 1])
assert c.status() == (0, -1)
"""


@pytest.mark.parametrize("T", [1, 80])
def test_first_call_of_a_process_is_captured(N, T):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", FIRST.format(root=root, T=T)], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]


@pytest.mark.parametrize("blocks", [1, 2, 3, 4, 5])
def test_repeated_calls_agree(N, blocks):
    """Rows of the same number of blocks (and neighbours of others), call after call: a
    pair's tiles change rows at every parity."""
    import torch
    rng = np.random.default_rng(blocks)
    k = np.where(rng.random(260) < 0.8, 64 * blocks - rng.integers(0, 64, 260), rng.integers(0, 400, 260))
    c = Case(N, [int(x) for x in k], H=128, topk=512, seed=blocks, seqs=[int(x) for x in rng.integers(0, 5, 260)]).build().call()
    c.check(rows=range(0, 260, 13))
    out, lse = c.d["out"].clone(), c.d["lse"].clone()
    for _ in range(40):
        c.d["out"].fill_(7.0)
        c.d["out"][c.T:] = 55.0
        c.call()
        assert torch.equal(c.d["out"], out) and torch.equal(c.d["lse"], lse)
    assert c.status() == (0, -1)
