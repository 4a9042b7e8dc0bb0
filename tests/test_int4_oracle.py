"""Pins of the packed 4-bit latent rows and of the batch plan's oracle (CPU)."""
import numpy as np
import pytest
import torch

from long_context_sparse_04_b200 import inputs as I
from oracle import dsa_ref as R


def test_scale_bytes_are_fp16_patterns():
    codes = np.arange(0xF8)
    f16 = torch.from_numpy((codes << 7).astype(np.int16)).view(torch.float16).double().numpy()
    np.testing.assert_array_equal(R.int4_scale_decode(codes), f16)
    # every scale times every code has at most 8 significant bits: exact in bf16
    v = R.int4_scale_decode(codes)[:, None] * np.arange(-8, 8)[None]
    np.testing.assert_array_equal(torch.from_numpy(v).to(torch.bfloat16).double().numpy(), v)
    # and so are 136 S and the terms of code * S = (136 + code) S - 136 S
    v = 136 * R.int4_scale_decode(codes)
    np.testing.assert_array_equal(torch.from_numpy(v).to(torch.bfloat16).double().numpy(), v)


def test_scale_encode_rounds_to_nearest_even():
    grid = R.int4_scale_decode(np.arange(0xF8))
    np.testing.assert_array_equal(R.int4_scale_encode(grid), np.arange(0xF8))
    mid = (grid[1:] + grid[:-1]) / 2
    got = R.int4_scale_encode(mid)
    assert (got % 2 == 0).all() and (np.abs(got.astype(int) - np.arange(1, 0xF8)) <= 1).all()
    np.testing.assert_array_equal(R.int4_scale_encode(np.nextafter(mid, 0)), np.arange(0xF7))
    np.testing.assert_array_equal(R.int4_scale_encode(np.nextafter(mid, np.inf)), np.arange(1, 0xF8))
    assert R.int4_scale_encode(np.array([1e30]))[0] == 0xF7


@pytest.mark.parametrize("d_c,d_r", [(512, 64), (64, 16), (32, 0), (96, 8), (512, 128)])
def test_pack_and_unpack(d_c, d_r):
    rng = np.random.default_rng(d_c + d_r)
    x = rng.standard_normal((40, d_c + d_r)) * np.exp(rng.uniform(-8, 8, (40, 1)))
    bits = I.to_bf16_bits(x.astype(np.float32))
    rows = R.int4_pack(bits, d_c, d_r)
    assert rows.shape[1] == R.int4_row_bytes(d_c, d_r) and rows.shape[1] % 16 == 0
    v, x = R.int4_unpack(rows, d_c, d_r), R.bf16_decode(bits)
    np.testing.assert_array_equal(v[:, d_c:], x[:, d_c:])          # RoPE: bit copy
    # half a step of the group's scale, and up to a sixteenth of the largest
    # value where the scale was rounded down
    g = x[:, :d_c].reshape(40, -1, 16)
    s = R.int4_scale_decode(rows[:, d_c // 2 + 2 * d_r: d_c // 2 + 2 * d_r + d_c // 16])[:, :, None]
    err = np.abs(v[:, :d_c].reshape(g.shape) - g)
    assert (err <= np.maximum(s / 2, np.abs(g).max(2, keepdims=True) / 16 + 1e-12)).all()
    assert np.sqrt(np.mean(err ** 2)) < 0.12 * np.sqrt(np.mean(g ** 2))
    # packing what was read gives the same bytes where the largest code is 7
    again = R.int4_pack(I.to_bf16_bits(v.astype(np.float32)), d_c, d_r)
    full = (np.abs(v[:, :d_c].reshape(g.shape)).max(2) == 7 * s[:, :, 0]).all(1)
    np.testing.assert_array_equal(again[full], rows[full])


def test_zero_and_tiny_groups():
    bits = I.to_bf16_bits(np.array([[0.0] * 16 + [2.0 ** -30] * 16], np.float32))
    rows = R.int4_pack(bits, 32, 0)
    assert not rows.any()


def _state(rng, B, P, W):
    lens = rng.integers(0, W * P // 2, B)
    held = -(-lens // P)
    pages = rng.permutation(int(held.sum()) + 40)
    table = np.full((B, W), -1)
    o = 0
    for b in range(B):
        table[b, : held[b]] = pages[o: o + held[b]]
        o += held[b]
    return lens, table, pages[o:].tolist(), len(pages)


@pytest.mark.parametrize("seed", range(8))
def test_plan_keeps_every_page_once(seed):
    """Over several steps, each page is in the free list or in one table entry."""
    rng = np.random.default_rng(seed)
    B, P, W = 13, int(rng.choice([1, 7, 16])), 30
    lens, table, free, num_pages = _state(rng, B, P, W)
    for _ in range(6):
        rel = rng.random(B) < 0.2
        n_new = np.where(rel, 0, rng.integers(0, 3 * P + 2, B))
        r = R.batch_plan(lens, n_new, rel, free, table, P, num_pages, 50)
        held = [p for b in range(B) for p in r["block_table"][b, : -(-r["seq_len"][b] // P)]]
        assert sorted(held + r["free_list"]) == list(range(num_pages))
        assert r["totals"][0] == r["start"][-1] == len(r["rows"]) <= 50
        slots = [s for _, _, s in r["rows"]]
        assert len(set(slots)) == len(slots) and all(s >= 0 for s in slots)
        for b, pos, s in r["rows"]:
            assert s == r["block_table"][b, pos // P] * P + pos % P
        lens, table, free = np.array(r["seq_len"]), r["block_table"], r["free_list"]


def test_plan_matches_the_plain_form():
    """The sequential rule against the prefix sums of the measured plain form."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")
    spec = importlib.util.spec_from_file_location("operators_plain", path)
    O = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(O)
    O.DEV = "cpu"
    for k, case in enumerate([
            dict(op="plan", seqs=23, lo=0, hi=40, ctx=300, page=16, pad=0, free=9, release=0.3),
            dict(op="plan", seqs=7, lo=1, hi=9, ctx=64, page=48, pad=30, free=2, release=0.0),
            dict(op="plan", seqs=1, lo=1, hi=1, ctx=64, page=64, pad=2, free=8, release=0.0)]):
        s = O.prepare(case, k)
        table, free = s["block_table"].clone().numpy(), s["free_pages"].tolist()[: case["free"]]
        got = O.run(s)
        want = R.batch_plan(s["seq_len"].tolist(), s["n_new"].tolist(), s["release_flags"].tolist(), free, table,
                            case["page"], s["num_pages"], s["max_tokens"])
        assert got["seq_len_out"].tolist() == want["seq_len"]
        assert got["tok_start"].tolist() == want["start"]
        assert got["totals"].tolist() == want["totals"]
        n = len(want["rows"])
        assert list(zip(got["row_seq"].tolist(), got["tok_pos"].tolist(), got["slot"].tolist()))[:n] == want["rows"]
        np.testing.assert_array_equal(got["block_table"].numpy(), want["block_table"])
        assert got["free_pages"].tolist()[: int(got["free_count_out"])] == want["free_list"]


@pytest.mark.parametrize("plant", ["nibble_order", "ceil_scale", "no_clip", "pop_bottom"])
def test_planted_mistakes_are_seen(plant, monkeypatch):
    """A wrong oracle fails a pin above."""
    if plant == "nibble_order":
        real = R.int4_unpack
        monkeypatch.setattr(R, "int4_unpack", lambda r, c, d: real(r, c, d)[:, np.arange(c + d) ^ (np.arange(c + d) < c)])
        with pytest.raises(AssertionError):
            test_pack_and_unpack(64, 16)
    elif plant == "ceil_scale":
        real = R.int4_scale_encode
        monkeypatch.setattr(R, "int4_scale_encode", lambda r: np.minimum(real(r) + (R.int4_scale_decode(real(r)) < r), 0xF7).astype(np.uint8))
        with pytest.raises(AssertionError):
            test_scale_encode_rounds_to_nearest_even()
    elif plant == "no_clip":
        real = R.int4_quantise
        monkeypatch.setattr(R, "int4_quantise", lambda c: (real(c)[0] + 1, real(c)[1]))
        with pytest.raises(AssertionError):
            test_pack_and_unpack(64, 16)
    else:
        real = R.batch_plan
        monkeypatch.setattr(R, "batch_plan", lambda a, b, c, free, *r, **k: real(a, b, c, list(free)[::-1], *r, **k))
        with pytest.raises(AssertionError):
            test_plan_matches_the_plain_form()
