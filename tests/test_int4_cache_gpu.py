"""The packed 4-bit latent cache on the GPU: every byte that dsa_cache_append and
dsa_cache_append_slots write, and every value that dsa_cache_read returns, equals
the oracle's (the codes and scales are integer decisions taken in fp32 on both
sides; the values are exact in bf16, and a key's is one fp32 product)."""
import numpy as np
import pytest

from long_context_sparse_04_b200 import inputs as I
from oracle import dsa_ref as R

pytestmark = pytest.mark.gpu
GUARD = 3          # rows behind the last that must stay as they are


@pytest.fixture(scope="module")
def N():
    from long_context_sparse_04_b200 import build
    build.build()
    from long_context_sparse_04_b200 import _native
    return _native


def dims(N, d_c=512, d_r=64, d_idx=128, mla=None, fp8=True):
    return N.dsa_dims(n_idx_heads=64, d_idx=d_idx, n_heads=128, d_c=d_c, d_r=d_r, topk=64,
                      idx_dtype=N.DSA_FP8_E4M3 if fp8 else N.DSA_F32, mla_dtype=N.DSA_INT4 if mla is None else mla,
                      sm_scale=1.0, algo=0)


class Cache:
    def __init__(self, N, d, tokens, fill=0xA5, table=None, page=64, num_seqs=1):
        import torch
        self.N, self.torch, self.d = N, torch, d
        self.row = N.dsa_latent_row_bytes(d)
        self.fp8 = d.idx_dtype == N.DSA_FP8_E4M3
        kb = d.d_idx * (1 if self.fp8 else 4)
        self.latent = torch.full((tokens, self.row), fill, dtype=torch.uint8, device="cuda")
        self.idx_k = torch.full((tokens, kb), fill, dtype=torch.uint8, device="cuda")
        self.scale = torch.full((tokens,), 0.5, device="cuda")
        self.table = None if table is None else torch.as_tensor(np.asarray(table, np.int32)).cuda()
        self.c = N.dsa_cache(latent=self.latent.data_ptr(), idx_k=self.idx_k.data_ptr(), idx_k_scale=self.scale.data_ptr(),
                             block_table=None if table is None else self.table.data_ptr(), page_size=page if table is not None else 0,
                             max_pages_per_seq=self.table.shape[1] if table is not None else 0, num_seqs=num_seqs, num_tokens=tokens)
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def args(self):
        return self.ws.data_ptr(), 256, self.torch.cuda.current_stream().cuda_stream

    def status(self):
        return self.N.dsa_read_device_status(self.ws.data_ptr(), self.args()[2])

    def bytes(self):
        return self.latent.cpu().numpy(), self.idx_k.cpu().numpy(), self.scale.cpu().numpy()


_ALIVE = []


def dev(x):
    """A device copy that lives to the end of the test (calls get its pointer)."""
    import torch
    x = np.ascontiguousarray(x)
    _ALIVE.append(torch.from_numpy(x.view(np.int16) if x.dtype == np.uint16 else x).cuda())
    return _ALIVE[-1]


@pytest.fixture(autouse=True)
def _free():
    yield
    _ALIVE.clear()


def special_latents(n, d_c, d_r, rng):
    """bf16 rows over many binades, with rows that reach the rule's corners: zeros,
    scales that tie, underflow, saturate and are subnormal, codes that tie, signed
    zeros, the largest bf16."""
    x = (rng.standard_normal((n, d_c + d_r)) * np.exp(rng.uniform(-14, 14, (n, 1)))).astype(np.float32)
    grid = R.int4_scale_decode(np.arange(R.INT4_SCALE_MAX + 1))
    mids = 7 * (grid[1:] + grid[:-1]) / 2                      # amax whose quotient ties (exact in bf16)
    if n > 8:
        x[0] = 0
        x[1] = -0.0
        x[2, :d_c] = 0
        x[2, : d_c: 16] = mids[60: 60 + d_c // 16]
        x[3, :d_c] = rng.integers(-15, 16, d_c) / 2            # codes that tie at scale 1
        x[3, : d_c: 16] = 7
        x[4, :d_c] = rng.standard_normal(d_c) * 2.0 ** -16     # subnormal and zero scales
        x[5, :d_c] = 2.0 ** -19 * rng.choice([-1, 1], d_c)
        x[6, :d_c] = rng.standard_normal(d_c) * 3e38 / 4       # scales that saturate
        x[7, :d_c] = 0
        x[7, : d_c: 16] = mids[: d_c // 16]                    # ties among the subnormal scales
    return I.to_bf16_bits(x)


def keys(n, d, rng):
    k = (rng.standard_normal((n, d)) * np.exp(rng.uniform(-20, 10, (n, 1)))).astype(np.float32)
    k[0] = 0
    return k


@pytest.mark.parametrize("n", [1, 2, 31, 1000])
@pytest.mark.parametrize("d_c,d_r,d_idx,fp8", [(512, 64, 128, True), (64, 16, 36, False), (32, 0, 512, True), (96, 264, 4, True)])
def test_append_by_slot_then_read(N, n, d_c, d_r, d_idx, fp8):
    import torch
    rng = np.random.default_rng(n + d_c)
    d, tokens = dims(N, d_c, d_r, d_idx, fp8=fp8), 2 * n + 5
    c = Cache(N, d, tokens)
    lat0, k0, s0 = (x.copy() for x in c.bytes())
    slot = rng.permutation(tokens)[:n].astype(np.int64)
    skip = rng.random(n) < 0.2
    slot[skip] = -1 - (np.arange(n)[skip] % 3)
    k, lat = keys(n, d_idx, rng), special_latents(n, d_c, d_r, rng)
    dk, dl, ds = dev(k), dev(lat), dev(slot)
    N.dsa_cache_append_slots(d, c.c, n, ds.data_ptr(), dk.data_ptr(), dl.data_ptr(), *c.args())
    go = slot >= 0
    lat0[slot[go]] = R.int4_pack(lat, d_c, d_r)[go]
    if fp8:
        codes, s = R.quantise_keys(k)
        k0[slot[go]], s0[slot[go]] = codes[go], s[go]
    else:
        k0[slot[go]] = k.view(np.uint8).reshape(n, -1)[go]
    got = c.bytes()
    np.testing.assert_array_equal(got[0], lat0)
    np.testing.assert_array_equal(got[1], k0)
    np.testing.assert_array_equal(got[2], s0)
    assert c.status() == (0, -1)
    # read: any order, repeats, holes, guard rows
    m = n + 7
    want = rng.integers(0, tokens, m).astype(np.int64)
    if n > 2:
        want = np.concatenate([slot[go], slot[go][:3], [-1]]).astype(np.int64) if go.any() else want
    m = len(want)
    ko = torch.full((m + GUARD, d_idx), 77.0, device="cuda")
    lo = torch.full((m + GUARD, d_c + d_r), 77.0, dtype=torch.bfloat16, device="cuda")
    N.dsa_cache_read(d, c.c, m, dev(want).data_ptr(), ko.data_ptr(), lo.data_ptr(), *c.args())
    lw = np.full((m + GUARD, d_c + d_r), 77.0)
    kw = np.full((m + GUARD, d_idx), 77.0, np.float32)
    ok = np.flatnonzero(want >= 0)
    lw[ok] = R.int4_unpack(lat0[want[ok]], d_c, d_r)
    if fp8:
        kw[ok] = R.e4m3_decode(k0[want[ok]]).astype(np.float32) * s0[want[ok]][:, None]
    else:
        kw[ok] = k0[want[ok]].view(np.float32)
    np.testing.assert_array_equal(lo.double().cpu().numpy(), lw)
    np.testing.assert_array_equal(ko.cpu().numpy(), kw)
    assert c.status() == (0, -1)
    assert N.dsa_read_kernel_trace(c.ws.data_ptr(), c.args()[2]) == N.DSA_KERNEL_CACHE_APPEND | N.DSA_KERNEL_CACHE_READ


def test_every_scale_and_tie(N):
    """Every finite bf16 as a group's largest value, with every tie of its scale."""
    amax = R.bf16_decode(np.arange(1, 0x7F80, dtype=np.uint16)).astype(np.float64)
    s = R.int4_scale_decode(R.int4_scale_encode((amax.astype(np.float32) / np.float32(7))))
    g = np.zeros((len(amax), 16))
    g[:, 0] = amax * np.where(np.arange(len(amax)) % 2, 1, -1)
    for j in range(7):                                         # (j + 1/2) scale: exact in bf16, below amax or clipped to it
        g[:, 1 + j] = np.minimum((j + 0.5) * s, amax)
        g[:, 8 + j] = -np.minimum(np.nextafter(np.float32(1), np.float32(2)) * (j + 0.5) * s * (1 + 2.0 ** -7), amax)
    g[:, 15] = np.minimum(s * 0.25, amax)
    rows = -(-len(amax) // 32)
    lat = np.zeros((rows, 512), np.float32)
    lat.reshape(-1)[: g.size] = g.reshape(-1)
    bits = I.to_bf16_bits(lat)
    d = dims(N, 512, 0, 4)
    c = Cache(N, d, rows)
    N.dsa_cache_append_slots(d, c.c, rows, dev(np.arange(rows, dtype=np.int64)).data_ptr(), None, dev(bits).data_ptr(), *c.args())
    np.testing.assert_array_equal(c.bytes()[0], R.int4_pack(bits, 512, 0))
    assert c.status() == (0, -1)


def test_keys_at_the_borders_of_e4m3(N):
    """Keys whose quotient lies on, or a unit in the last place beside, every border
    between two e4m3 codes, under scales of many magnitudes."""
    rng = np.random.default_rng(2)
    vals = np.unique(np.abs(R.e4m3_decode(np.arange(127, dtype=np.uint8)))).astype(np.float64)
    mids = (vals[1:] + vals[:-1]) / 2
    scales = np.exp(rng.uniform(-80, 80, 300)).astype(np.float32)
    scales[:4] = [1e-40, 1.0, 3e-39, 2.0 ** -149 * 3]
    k = np.zeros((len(scales), 508), np.float32)
    for r, s in enumerate(scales):
        m = (mids * np.float64(s)).astype(np.float32)
        row = np.concatenate([m, np.nextafter(m, np.float32(np.inf)), np.nextafter(m, np.float32(0)), -m])
        k[r, : len(row)] = row
        k[r, -1] = np.float32(448) * s
    k = np.where(np.isfinite(k), k, 0).astype(np.float32)
    d = dims(N, 32, 0, 508)
    c = Cache(N, d, len(scales))
    N.dsa_cache_append_slots(d, c.c, len(scales), dev(np.arange(len(scales), dtype=np.int64)).data_ptr(), dev(k).data_ptr(),
                             None, *c.args())
    codes, s = R.quantise_keys(k)
    got = c.bytes()
    np.testing.assert_array_equal(got[1], codes)
    np.testing.assert_array_equal(got[2], s)


def test_every_byte_reads_as_its_value(N):
    """All 16 codes at all 256 scale bytes, those the writers never use among them."""
    import torch
    d = dims(N, 512, 0, 4)
    c = Cache(N, d, 256)
    rows = np.zeros((256, c.row), np.uint8)
    rows[:, :256] = np.random.default_rng(0).integers(0, 256, (256, 256))
    rows[:, :64] = np.tile(np.arange(0, 256, 4, dtype=np.uint8), (256, 1))
    rows[:, 256:288] = np.arange(256, dtype=np.uint8)[:, None]
    c.latent.copy_(torch.from_numpy(rows))
    lo = torch.empty((256, 512), dtype=torch.bfloat16, device="cuda")
    N.dsa_cache_read(d, c.c, 256, dev(np.arange(256, dtype=np.int64)).data_ptr(), None, lo.data_ptr(), *c.args())
    np.testing.assert_array_equal(lo.double().cpu().numpy(), R.int4_unpack(rows, 512, 0))


@pytest.mark.parametrize("mla", ["bf16", "f32", "int4"])
def test_one_cache_alone(N, mla):
    """k_new or latent_new NULL leaves the other cache as it is; slots write the
    uncompressed caches too."""
    import torch
    rng = np.random.default_rng(4)
    m = {"bf16": N.DSA_BF16, "f32": N.DSA_F32, "int4": N.DSA_INT4}[mla]
    d, n = dims(N, mla=m), 50
    c = Cache(N, d, 64)
    lat0, k0, s0 = (x.copy() for x in c.bytes())
    slot = rng.permutation(64)[:n].astype(np.int64)
    if mla == "f32":
        lat = rng.standard_normal((n, 576)).astype(np.float32)
        packed = lat.view(np.uint8).reshape(n, -1)
    else:
        lat = special_latents(n, 512, 64, rng)
        packed = R.int4_pack(lat, 512, 64) if mla == "int4" else lat.view(np.uint8).reshape(n, -1)
    k = keys(n, 128, rng)
    N.dsa_cache_append_slots(d, c.c, n, dev(slot).data_ptr(), None, dev(lat).data_ptr(), *c.args())
    lat0[slot] = packed
    for a, b in zip(c.bytes(), (lat0, k0, s0)):
        np.testing.assert_array_equal(a, b)
    N.dsa_cache_append_slots(d, c.c, n, dev(slot).data_ptr(), dev(k).data_ptr(), None, *c.args())
    k0[slot], s0[slot] = R.quantise_keys(k)
    for a, b in zip(c.bytes(), (lat0, k0, s0)):
        np.testing.assert_array_equal(a, b)
    ko = torch.zeros((n, 128), device="cuda")
    lo = torch.zeros((n, 576), dtype=torch.float32 if mla == "f32" else torch.bfloat16, device="cuda")
    N.dsa_cache_read(d, c.c, n, dev(slot).data_ptr(), ko.data_ptr(), None, *c.args())
    N.dsa_cache_read(d, c.c, n, dev(slot).data_ptr(), None, lo.data_ptr(), *c.args())
    np.testing.assert_array_equal(ko.cpu().numpy(), R.e4m3_decode(k0[slot]).astype(np.float32) * s0[slot][:, None])
    want = lat if mla == "f32" else R.int4_unpack(packed, 512, 64) if mla == "int4" else R.bf16_decode(lat)
    np.testing.assert_array_equal(lo.double().cpu().numpy(), want.astype(np.float64))
    assert c.status() == (0, -1)


@pytest.mark.parametrize("by", ["slot", "position"])
@pytest.mark.parametrize("kind", ["nan", "inf", "key", "range"])
def test_one_bad_token(N, by, kind):
    """A token with a non-finite latent dim or key, or a destination outside the
    cache, is named and not written; a NaN in its RoPE dims is data."""
    rng = np.random.default_rng(9)
    n, bad, page = 40, 17, 64
    table = np.array([[2, 0], [3, 1]])
    d = dims(N)
    c = Cache(N, d, 4 * page, table=table if by == "position" else None, page=page, num_seqs=2)
    lat0, k0, s0 = (x.copy() for x in c.bytes())
    seq, pos = np.arange(n) % 2, np.arange(n) * 3
    slot = (table[seq, pos // page] * page + pos % page).astype(np.int64)
    k, lat = keys(n, 128, rng), special_latents(n, 512, 64, rng)
    lat[5, 520] = 0x7FC0                                        # RoPE NaN: copied
    code = N.DSA_ERR_INVALID_ARG
    if kind == "nan":
        lat[bad, 511] = 0x7FC1
    elif kind == "inf":
        lat[bad, 0] = 0xFF80
    elif kind == "key":
        k[bad, 127] = np.inf
    elif by == "slot":
        slot[bad], code = 4 * page, N.DSA_ERR_OUT_OF_RANGE
    else:
        pos[bad], code = 2 * page, N.DSA_ERR_OUT_OF_RANGE
    if by == "slot":
        N.dsa_cache_append_slots(d, c.c, n, dev(slot).data_ptr(), dev(k).data_ptr(), dev(lat).data_ptr(), *c.args())
    else:
        N.dsa_cache_append(d, c.c, n, dev(seq.astype(np.int32)).data_ptr(), dev(pos.astype(np.int32)).data_ptr(),
                           dev(k).data_ptr(), dev(lat).data_ptr(), *c.args())
    assert c.status() == (code, bad)
    go = np.arange(n) != bad
    lat_ok, k_ok = lat.copy(), k.copy()
    lat_ok[bad], k_ok[bad] = 0, 0
    lat0[slot[go]] = R.int4_pack(lat_ok, 512, 64)[go]
    codes, s = R.quantise_keys(k_ok)
    k0[slot[go]], s0[slot[go]] = codes[go], s[go]
    for a, b in zip(c.bytes(), (lat0, k0, s0)):
        np.testing.assert_array_equal(a, b)


def test_read_names_a_slot_outside(N):
    import torch
    d = dims(N)
    c = Cache(N, d, 64, fill=0)
    lo = torch.full((9, 576), 77.0, dtype=torch.bfloat16, device="cuda")
    slot = np.arange(9, dtype=np.int64)
    slot[4] = 64
    N.dsa_cache_read(d, c.c, 9, dev(slot).data_ptr(), None, lo.data_ptr(), *c.args())
    assert c.status() == (N.DSA_ERR_OUT_OF_RANGE, 4)
    assert (lo[4] == 77).all() and (lo[[0, 1, 2, 3, 5, 6, 7, 8]] == 0).all()
