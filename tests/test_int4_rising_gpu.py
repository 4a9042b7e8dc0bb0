"""The running maximum of the attention over packed rows: heads whose logits rise from
block to block, at rates that make the accumulator rescale in every block, every second
(always one softmax group) or every third (the groups in turn), beside heads that fall
or stay, in the same warps; with one, two and four key splits."""
import numpy as np
import pytest

from long_context_sparse_04_b200 import inputs as I
from tests.test_int4_mla_gpu import Case

pytestmark = pytest.mark.gpu

# a head's logits grow by this per block of 64 keys (natural log; the accumulator rescales
# when the maximum has grown by 8 ln 2 = 5.5 since it last did)
RATES = [6.0, 3.25, 2.0, 1.0, 0.0, -1.0, -6.0, 0.5, 7.5]


@pytest.fixture(scope="module")
def N():
    from long_context_sparse_04_b200 import build
    build.build()
    from long_context_sparse_04_b200 import _native
    return _native


def rising(N, T, keys, order, H=128, algo=0):
    c = Case(N, [keys] * T, H=H, seqs=[0] * T, page=64, seed=T, algo=algo)
    block = np.arange(keys) // 64                     # of a key within the selection
    if order == "last_block_first":
        block = (block.max() - block)
    elif order == "saw":                              # up, back down, up
        block = np.where(block % 5 == 4, 0, block)
    pos = np.arange(keys)
    rope = I.to_bf16_bits(block.astype(np.float32))   # whole numbers below 256: exact
    at = c.physical(0, pos)
    c.rows[at, 256] = rope & 0xFF                     # the first RoPE dim of each key
    c.rows[at, 257] = rope >> 8
    for t in range(T):
        c.idx[t, :keys] = pos
    rate = np.array([RATES[(h + h // 9) % 9] for h in range(H)], np.float32)
    c.q[:, :, 512] = I.to_bf16_bits(24 * rate)[None]  # sm_scale = 1/24: the logit of block j is j * rate and noise
    return c


@pytest.mark.parametrize("order", ["rising", "last_block_first", "saw"])
@pytest.mark.parametrize("T", [2, 21, 40, 80])
def test_rescale_in_every_pattern(N, T, order):
    c = rising(N, T, 2048, order).build().call()
    c.check(rows=[0, T // 2, T - 1])
    assert c.status() == (0, -1)


@pytest.mark.parametrize("keys", [65, 128, 129, 500, 1030])
@pytest.mark.parametrize("T", [3, 30, 90])
def test_ragged_rows(N, T, keys):
    rising(N, T, keys, "rising", H=72).build().call().check(rows=[0, T - 1])


def test_cuda_cores(N):
    rising(N, 4, 500, "saw", H=16, algo=N.DSA_ALGO_SIMT).build().call().check()
