"""lq_norm_block where the mean of squares is a float, and so is eps, but not their sum. Tolerances as in
test_gpu_norm_block."""
import numpy as np
import pytest
import torch

from tests.test_gpu_int8 import F32
from tests.test_gpu_norm_block import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,size,eps", [(1, 5e18, 3.4e38), (1, 1e18, 3.4e38), (2, 3e18, 3.39e38), (3, 6e18, 3.3e38)])
def test_eps_and_mean_pass_the_largest_float(K, size, eps):
    import bit_matmul_amd as lq
    run(lq, np.random.default_rng(K + 1), 9, K, F32, F32, F32, y=False, size=size, eps=eps)
    run(lq, np.random.default_rng(K + 1), 9, K, F32, F32, F32, h=False, post=True, size=size, eps=eps)
