"""Every scale byte of a packed row, those that the writers never use among them, has the
value that include/dsa.h states."""
import numpy as np
import pytest

from long_context_sparse_04_b200 import inputs as I
from oracle import dsa_ref as R


def stated(byte):
    e, m = byte >> 3, byte & 7
    return (8 + m) * 2.0 ** (e - 18) if e else m * 2.0 ** -17


def test_the_oracle_reads_every_byte_as_stated():
    np.testing.assert_array_equal(R.int4_scale_decode(np.arange(256)), [stated(b) for b in range(256)])
    assert stated(0xF8) == 65536 and stated(0xFF) == 122880


def test_the_header_states_the_values():
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = " ".join(open(os.path.join(root, "include", "dsa.h")).read().replace("*", " ").split())
    assert "(8 + m) 2^(e - 18), and m 2^-17 for e = 0" in text and "0xF8 to 0xFF are 65536 to 122880" in text


def rows_of(d_c, d_r, seed):
    """Scale bytes of the two top exponents, every code, a plain RoPE key."""
    rng = np.random.default_rng(seed)
    n = 64
    bits = I.to_bf16_bits(rng.standard_normal((n, d_c + d_r)).astype(np.float32))
    rows = R.int4_pack(bits, d_c, d_r)
    rows[:, : d_c // 2] = rng.integers(0, 256, (n, d_c // 2))
    at = d_c // 2 + 2 * d_r
    rows[:, at: at + d_c // 16] = rng.integers(0xF0, 0x100, (n, d_c // 16))
    return rows


@pytest.mark.gpu
def test_read_of_the_largest_scales():
    import torch
    from long_context_sparse_04_b200 import _native as N
    rows = rows_of(512, 64, 1)
    lat = torch.from_numpy(rows).cuda()
    slot, out = torch.arange(64, device="cuda"), torch.empty((64, 576), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    d = N.dsa_dims(n_idx_heads=64, d_idx=128, n_heads=128, d_c=512, d_r=64, topk=64, idx_dtype=N.DSA_FP8_E4M3, mla_dtype=N.DSA_INT4,
                   sm_scale=1.0, algo=0)
    st = torch.cuda.current_stream().cuda_stream
    N.dsa_cache_read(d, N.dsa_cache(latent=lat.data_ptr(), num_seqs=1, num_tokens=64), 64, slot.data_ptr(), None, out.data_ptr(),
                     ws.data_ptr(), 256, st)
    got = out.double().cpu().numpy()
    q = np.empty((64, 512))
    for i in range(8):                              # the codes, from the bytes
        w = np.ascontiguousarray(rows[:, :256]).view("<u4")
        v = ((w >> np.uint32(4 * (i // 2) + 16 * (i % 2))) & np.uint32(15)).astype(int)
        q[:, i::8] = np.where(v > 7, v - 16, v)
    scale = np.array([stated(b) for b in range(256)])[rows[:, 384:416]]
    np.testing.assert_array_equal(got[:, :512], q * np.repeat(scale, 16, axis=1))
    assert N.dsa_read_device_status(ws.data_ptr(), st) == (0, -1)


@pytest.mark.gpu
@pytest.mark.parametrize("algo", ["auto", "simt"])
@pytest.mark.parametrize("T", [2, 80])
def test_attention_over_the_largest_scales(T, algo):
    from long_context_sparse_04_b200 import _native as N
    from tests.test_int4_mla_gpu import Case
    a = {"auto": N.DSA_ALGO_AUTO, "simt": N.DSA_ALGO_SIMT}[algo]
    c = Case(N, [64, 130] * (T // 2), topk=128, seed=T, algo=a, q_std=2.0 ** -22)
    big = rows_of(512, 64, T)
    c.rows[:] = big[np.arange(len(c.rows)) % 64]
    c.build().call().check(rows=[0, 1, T - 1])
    assert c.status() == (0, -1)
