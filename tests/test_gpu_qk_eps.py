"""Heads' norms whose mean of squares is a float, and so is eps, but not their sum. Tolerances as in
test_gpu_qk_norm_rope."""
import numpy as np
import pytest
import torch

from tests.gpu_util import DEV, note
from tests.test_gpu_qk_norm_rope import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,size,eps", [(1, 1.5e19, 2e38), (1, 1e19, 3.4e38), (4, 8e18, 3e38), (3, 1e19, 3.3e38), (64, 2e18, 3.4e38),
                                          (1, 1.8e19, 1.6e37), (2, 1.0, 3.4e38)])
def test_eps_and_mean_pass_the_largest_float(dim, size, eps):
    import bit_matmul_amd as lq
    rng = np.random.default_rng(dim)
    x = torch.from_numpy((size * rng.choice([-1, 1], size=(5, 3, dim)) * rng.uniform(0.99, 1, (5, 3, dim))).astype(np.float32)).to(DEV)
    x[2, 1] *= 1e-3
    out = torch.empty_like(x)
    note(f"lq_qk_norm_rope dim={dim} values {size} eps={eps}")
    lq.lq_qk_norm_rope(None, None, q=x, q_out=out, eps=eps)
    torch.cuda.synchronize()
    check(out, x, np.zeros(5), np.zeros(0), None, True, False, eps, False)
