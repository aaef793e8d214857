"""lq_norm_block where the sum of squares passes the largest float: eps still counts, and small values next
to the large ones keep their accuracy. Tolerances as in test_gpu_norm_block."""
import numpy as np
import pytest
import torch

from tests.gpu_util import DEV, note
from tests.test_gpu_int8 import F32, U32, host64, randn
from tests.test_gpu_norm_block import norm_err, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lq():
    import bit_matmul_amd
    assert torch.cuda.is_available()
    return bit_matmul_amd


@pytest.mark.parametrize("K,size,eps", [(65536, 1e17, 1e34), (65536, 7e16, 1e30), (3000, 1e18, 1e36), (3000, 1e19, 1e38),
                                        (70, 2e19, 3e38), (1, 3e19, 1e38), (70, 1e25, 1e38), (1500, 1e18, 2e27)])
def test_large_eps_next_to_large_values(lq, K, size, eps):
    """The mean of squares may be as small as 4.6e33 where their sum overflows: eps is no less than that."""
    run(lq, np.random.default_rng(K), 2, K, F32, F32, F32, y=False, size=size, eps=eps)
    run(lq, np.random.default_rng(K), 2, K, F32, F32, F32, h=False, post=True, size=size, eps=eps)


@pytest.mark.parametrize("small", [1e-12, 1e-15, 1e-18])
@pytest.mark.parametrize("K", [4, 1030, 17000])
def test_small_values_next_to_large_ones(lq, K, small):
    """a = h / rms(h) w with weights that lift it: the norm's factor and the two products' roundings, of each
    value for itself (h / rms is a normal float: at least 1e-18 / 3e19)."""
    rng = np.random.default_rng(K)
    h = randn(rng, 2, K).abs() * small + small
    h[:, ::max(1, K // 7)] = 2e19
    w, a = torch.full((K,), 1e30, device=DEV), torch.empty(2, K, device=DEV)
    note(f"lq_norm_block small values K={K} {small}")
    lq.lq_norm_block(2, K, h=h, pre=True, w_pre=w, a=a)
    torch.cuda.synchronize()
    h64 = host64(h)
    want = h64 / np.sqrt(np.mean(h64 * h64, axis=1, keepdims=True) + float(np.float32(1e-5))) * float(np.float32(1e30))
    assert np.all(np.abs(host64(a) - want) <= np.abs(want) * (norm_err(K) + 2 * U32))
