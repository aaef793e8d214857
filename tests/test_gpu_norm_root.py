"""The mean of squares and its reciprocal root in lq_norm_block, as near as 32 bits allow: a row's values all
share their error, so that it is no noise that a product behind the norm would average out."""
import numpy as np
import pytest
import torch

from tests.gpu_util import DEV, note
from tests.test_gpu_int8 import U32, host64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lq():
    import bit_matmul_amd
    assert torch.cuda.is_available()
    return bit_matmul_amd


def normed(lq, h, post, eps=1e-30):
    B, K = h.shape
    a = torch.empty_like(h)
    note(f"lq_norm_block root B={B} K={K} post={post}")
    if post:
        lq.lq_norm_block(B, K, y=h, post=True, a=a, eps=eps)
    else:
        lq.lq_norm_block(B, K, h=h, pre=True, a=a, eps=eps)
    torch.cuda.synchronize()
    return host64(a)


@pytest.mark.parametrize("K", [1024, 16384])
@pytest.mark.parametrize("lead", [0, 3, 12])
@pytest.mark.parametrize("post", [False, True])
def test_sum_of_squares_in_short_chains(lq, K, lead, post):
    """A thread's 16 values: one is 1, the others' squares lie just below half a unit of its last place, so
    that a chain of 16 additions may lose all of them (15 roundings, 7.5 after the root). In four chains joined
    pairwise at most 3 are lost one after another and 2 additions round, each by 2^-24 at most; the threads'
    sums are equal and double exactly. Half of that after the root, and the root's own rounding: 3.5."""
    h = np.full((1, K), 2.0 ** -12 * 0.99, dtype=np.float32)
    block = np.arange(K) % 1024
    h[0, block % 512 % 8 + 8 * (block // 512) == lead] = 1.0
    want = 1.0 / np.sqrt(np.mean(h.astype(np.float64) ** 2))
    a = normed(lq, torch.from_numpy(h).to(DEV), post)[h == 1.0]
    assert np.all(np.abs(a / want - 1) <= 3.5 * U32), np.abs(a / want - 1).max() / U32


@pytest.mark.parametrize("post", [False, True])
def test_reciprocal_root_is_rounded_once(lq, post):
    """Rows of ones and whole numbers m in turn: every sum, and their mean (1 + m^2) / 2, is exact in 32 bits
    (8 (1 + m^2) in a thread is below 2^24), and eps vanishes in it. The values at the ones are 1 / sqrt of the
    mean itself: half a unit of the last place, and 2^-16 of that for the correction's own roundings (its
    residual of at most 2^-22 is off by 2^-45)."""
    m = np.arange(1, 1400, 2)
    h = np.ones((len(m), 1024), dtype=np.float32)
    h[:, 1::2] = m[:, None]
    a = normed(lq, torch.from_numpy(h).to(DEV), post)[:, 0::2]
    want = np.sqrt(2.0 / (1.0 + m.astype(np.float64) ** 2))[:, None]
    ulp = np.spacing(want.astype(np.float32)).astype(np.float64)
    assert np.all(np.abs(a - want) <= 0.5 * ulp * (1 + 2.0 ** -16)), (np.abs(a - want) / ulp).max()


@pytest.mark.parametrize("K", [5, 4099, 40000])
def test_roots_of_ordinary_rows(lq, K):
    """The error that a row's values share, at both ends of the range too: the thread's chain of C additions
    of four chains, 2 joins, 10 levels, halved, and the division's, eps' and the root's roundings."""
    C = 1 if K <= 16384 else 4
    bound = ((4 * C + 12) / 2 + 1 + 1) * U32
    rng = np.random.default_rng(K)
    for size in (1e-15, 1.0, 1e16):
        h = torch.from_numpy((rng.standard_normal((8, K)) * size).astype(np.float32)).to(DEV)
        a = normed(lq, h, False)
        h64 = host64(h)
        want = h64 / np.sqrt(np.mean(h64 * h64, axis=1, keepdims=True) + float(np.float32(1e-30)))
        assert np.all(np.abs(a - want) <= np.abs(want) * (bound + U32))
