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
