"""Host-side refusals and descriptors of the 4-bit cache calls and the batch plan
(CPU only: every call here is refused before any device work)."""
import ctypes
import os
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20


@pytest.fixture(scope="module")
def N():
    from long_context_sparse_04_b200 import build
    build.build()
    from long_context_sparse_04_b200 import _native
    return _native


def dims(N, **kw):
    d = dict(n_idx_heads=64, d_idx=128, n_heads=128, d_c=512, d_r=64, topk=2048,
             idx_dtype=N.DSA_FP8_E4M3, mla_dtype=N.DSA_INT4, sm_scale=1 / 24, algo=0)
    d.update(kw)
    return N.dsa_dims(**d)


def cache(N, **kw):
    d = dict(latent=FAKE, idx_k=FAKE, idx_k_scale=FAKE, seq_start=None, block_table=FAKE, page_size=64,
             max_pages_per_seq=8, num_seqs=3, num_tokens=64 * 10)
    d.update(kw)
    return N.dsa_cache(**d)


def plan(N, **kw):
    d = {n: FAKE for n, t in N.dsa_plan._fields_ if t is ctypes.c_void_p}
    d.update(free_capacity=10, max_tokens=7)
    d.update(kw)
    return N.dsa_plan(**d)


def test_plan_struct_matches_the_c_compiler(N):
    names = [n for n, _ in N.dsa_plan._fields_]
    prog = '#include <stdio.h>\n#include <stddef.h>\n#include "dsa.h"\nint main(void) {\n  printf("%zu", sizeof(dsa_plan));\n'
    prog += "".join(f'  printf(" %zu", offsetof(dsa_plan, {n}));\n' for n in names) + "  return 0;\n}\n"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        open(c, "w").write(prog)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = list(map(int, subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()))
    assert got == [ctypes.sizeof(N.dsa_plan)] + [getattr(N.dsa_plan, n).offset for n in names]


def test_row_bytes_and_workspaces(N):
    from oracle import dsa_ref as R
    for d_c, d_r in ((512, 64), (64, 16), (32, 0), (96, 8)):
        assert N.dsa_latent_row_bytes(dims(N, d_c=d_c, d_r=d_r)) == R.int4_row_bytes(d_c, d_r)
    assert N.dsa_latent_row_bytes(dims(N, mla_dtype=N.DSA_BF16)) == 1152
    assert N.dsa_latent_row_bytes(dims(N, mla_dtype=N.DSA_F32)) == 2304
    assert N.dsa_workspace_size(dims(N), None, N.DSA_OP_CACHE_READ) == 256
    assert N.dsa_workspace_size(None, None, N.DSA_OP_BATCH_PLAN) == 256
    for bad in (dict(d_c=48), dict(d_c=544), dict(d_r=4, d_c=64)):
        assert N.dsa_latent_row_bytes(dims(N, **bad)) == 0, bad
        assert N.dsa_workspace_size(dims(N, **bad), None, N.DSA_OP_CACHE_READ) == 0, bad
    assert N.dsa_latent_row_bytes(dims(N, mla_dtype=N.DSA_FP8_E4M3)) == 0


@pytest.mark.parametrize("call", ["append", "read"])
def test_slot_calls_refuse(N, call):
    def run(d=None, c=None, n=5, slot=FAKE, k=FAKE, lat=FAKE, ws=FAKE, nb=256):
        f = N.dsa_cache_append_slots if call == "append" else N.dsa_cache_read
        return f(d or dims(N), c or cache(N), n, slot, k, lat, ws, nb, None, check=False)

    inv, uns, wsp = N.DSA_ERR_INVALID_ARG, N.DSA_ERR_UNSUPPORTED, N.DSA_ERR_WORKSPACE
    assert run(d=dims(N, d_c=48)) == uns
    assert run(n=-1) == inv
    assert run(slot=None) == inv
    assert run(slot=FAKE + 4) == inv
    assert run(k=None, lat=None) == inv
    assert run(k=FAKE + 4) == inv
    assert run(lat=FAKE + 8) == inv
    assert run(c=cache(N, latent=None)) == inv
    assert run(c=cache(N, idx_k=None)) == inv
    assert run(c=cache(N, idx_k_scale=None)) == inv
    assert run(c=cache(N, latent=FAKE + 16)) == inv
    assert run(c=cache(N, num_tokens=100)) == inv
    assert run(ws=None) == wsp
    assert run(nb=255) == wsp
    assert run(ws=FAKE + 16) == wsp
    assert run(n=0, slot=None, k=None, lat=None, c=cache(N, latent=None, idx_k=None)) == N.DSA_OK
    if call == "append":
        assert run(d=dims(N, d_idx=516)) == uns
    with pytest.raises(N.DSAError):
        N.dsa_cache_read(dims(N), cache(N), -1, FAKE, FAKE, FAKE, FAKE, 256, None)


def test_plan_refuses(N):
    def run(c=None, p=None, ws=FAKE, nb=256):
        return N.dsa_batch_plan(c or cache(N), p or plan(N), ws, nb, None, check=False)

    inv, uns, wsp = N.DSA_ERR_INVALID_ARG, N.DSA_ERR_UNSUPPORTED, N.DSA_ERR_WORKSPACE
    for name in ("seq_len", "n_new", "seq_len_out", "tok_start", "totals", "row_seq", "row_klen", "tok_pos", "slot",
                 "free_count", "free_count_out", "free_pages"):
        assert run(p=plan(N, **{name: None})) == inv, name
    assert run(p=plan(N, max_tokens=-1)) == inv
    assert run(p=plan(N, free_capacity=9)) == inv
    assert run(p=plan(N, slot=FAKE + 4)) == inv
    assert run(c=cache(N, num_seqs=0)) == inv
    assert run(c=cache(N, page_size=0)) == inv
    assert run(c=cache(N, num_tokens=100)) == inv
    assert run(c=cache(N, max_pages_per_seq=0)) == inv
    assert run(c=cache(N, num_seqs=16385)) == uns
    assert run(c=cache(N, num_seqs=16384, max_pages_per_seq=1 << 17)) == uns
    assert run(ws=None) == wsp
    assert run(nb=0) == wsp
    assert N.LIB.dsa_batch_plan(None, None, FAKE, 256, None) == inv


def test_attention_over_int4_refuses(N):
    rows = N.dsa_rows(num_rows=4, row_seq=FAKE, row_klen=FAKE, max_klen=100, q_group=1)
    f = lambda **kw: N.dsa_sparse_mla_fwd(dims(N, **kw), rows, cache(N), FAKE, FAKE, FAKE, None, FAKE, 1 << 30,  # noqa: E731
                                          None, check=False)
    assert f(d_c=48) == N.DSA_ERR_UNSUPPORTED
    assert f(d_c=1024) == N.DSA_ERR_UNSUPPORTED
    assert f(mla_dtype=N.DSA_FP8_E4M3) == N.DSA_ERR_INVALID_ARG
    assert f(mla_dtype=4) == N.DSA_ERR_INVALID_ARG
    assert N.dsa_sparse_mla_fwd(dims(N), rows, cache(N), FAKE + 8, FAKE, FAKE, None, FAKE, 1 << 30, None,
                                check=False) == N.DSA_ERR_INVALID_ARG
