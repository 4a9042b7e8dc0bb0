"""The CUDA-core attention reads nothing for a row of no sequence, in any type."""
import numpy as np
import pytest

from long_context_sparse_04_b200 import inputs as I
from oracle import dsa_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [3, -1, 2 ** 31 - 1])
@pytest.mark.parametrize("layout", ["paged", "starts", "one"])
@pytest.mark.parametrize("mla", ["bf16", "f32", "int4"])
def test_skipped_and_named(mla, layout, bad):
    import torch
    from long_context_sparse_04_b200 import _native as N
    rng = np.random.default_rng(4)
    B, H, d_c, d_r, topk, tokens = 3, 8, 64, 16, 40, 384
    T = 4
    kv = I.to_bf16_bits(rng.standard_normal((tokens, d_c + d_r)).astype(np.float32))
    q = I.to_bf16_bits((rng.standard_normal((T, H, d_c + d_r)) * 0.3).astype(np.float32))
    val = R.bf16_decode(kv).astype(np.float64)
    if mla == "int4":
        rows = R.int4_pack(kv, d_c, d_r)
        val = R.int4_unpack(rows, d_c, d_r)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    f32 = mla == "f32"
    lat = dev(rows) if mla == "int4" else dev(val.astype(np.float32)) if f32 else dev(kv.view(np.int16))
    qd = dev(R.bf16_decode(q).astype(np.float32)) if f32 else dev(q.view(np.int16))
    idx = np.stack([np.sort(rng.permutation(100)[:topk]) for _ in range(T)]).astype(np.int32)
    seq = np.array([0, 1, bad, 2], np.int32)
    table, starts = np.array([[4, 1], [0, 5], [3, 2]], np.int32), np.array([10, 150, 280], np.int32)
    dt = torch.float32 if f32 else torch.bfloat16
    out = torch.full((T + 1, H, d_c), 5.0, dtype=dt, device="cuda")
    lse = torch.full((T + 1, H), 5.0, device="cuda")
    d = N.dsa_dims(n_idx_heads=64, d_idx=128, n_heads=H, d_c=d_c, d_r=d_r, topk=topk, idx_dtype=N.DSA_FP8_E4M3,
                   mla_dtype={"bf16": N.DSA_BF16, "f32": N.DSA_F32, "int4": N.DSA_INT4}[mla], sm_scale=0.125, algo=N.DSA_ALGO_SIMT)
    keep = [dev(x) for x in (seq, np.full(T, 100, np.int32), idx, table, starts)]
    ptr = [x.data_ptr() for x in keep]
    kw = dict(paged=dict(block_table=ptr[3], page_size=64, max_pages_per_seq=2), starts=dict(seq_start=ptr[4]), one={})[layout]
    cache = N.dsa_cache(latent=lat.data_ptr(), num_seqs=B, num_tokens=tokens, **kw)
    r = N.dsa_rows(num_rows=T, row_seq=ptr[0], row_klen=ptr[1], max_klen=100, q_group=1)
    nb = N.dsa_workspace_size(d, r, N.DSA_OP_SPARSE_MLA)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    N.dsa_sparse_mla_fwd(d, r, cache, qd.data_ptr(), ptr[2], out.data_ptr(), lse.data_ptr(), ws.data_ptr(), nb, st)
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    code = N.dsa_read_device_status(ws.data_ptr(), st)
    assert code == ((0, -1) if layout == "one" else (N.DSA_ERR_OUT_OF_RANGE, 2))
    for t in range(T):
        if t == 2 and layout != "one":
            assert (o[t] == 0).all() and np.isneginf(l[t]).all()
            continue
        at = table[seq[t], idx[t] // 64] * 64 + idx[t] % 64 if layout == "paged" else idx[t] + (starts[seq[t]] if layout == "starts" else 0)
        ro, rl = R.sparse_mla_row(R.bf16_decode(q[t]).astype(np.float64), val[at], d_c, 0.125)
        # fp32 sums of 40 keys and 80 dims, logits below 8: 2^-24 (2 * 80 * 8 + 2 * 40) < 2^-13, and half a
        # step of the output's type (2^-8 of a value below 8 at most)
        tol = 2.0 ** -13 * (1 + np.abs(val[at]).max()) + (0 if f32 else 2.0 ** -8 * np.abs(ro))
        assert (np.abs(o[t] - ro) <= tol).all() and (np.abs(l[t] - rl) <= 2.0 ** -13).all()
    assert (o[T] == 5).all() and (l[T] == 5).all()
