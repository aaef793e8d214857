"""4-bit rows with T are those of the header's v to the bit: c x and the power of two, each rounded once, sums and
differences in fp32 stage by stage from neighbours to the farthest values, sqrt(2) where log2 hb is odd. (A sum of two
floats has one rounding, so the same stages on the CPU give the same floats.)"""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_mx4 import BF, DEV, F32, quant, randn, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lq():
    import bit_matmul_amd
    assert torch.cuda.is_available()
    return bit_matmul_amd


def stages(x, c, hb):
    """T x in fp32."""
    v = x.astype(np.float32)
    v = v if c is None else v * c
    log = int(math.log2(hb))
    v = v * np.float32(2.0 ** -((log + 1) // 2))
    h = 1
    while h < hb:
        p = v.reshape(v.shape[0], -1, 2, h)
        v = np.stack((p[:, :, 0] + p[:, :, 1], p[:, :, 0] - p[:, :, 1]), axis=2)
        h *= 2
    v = v.reshape(x.shape)
    assert v.dtype == np.float32
    return v * np.float32(math.sqrt(2.0)) if log % 2 else v


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("hb", [2, 4, 8, 16, 32, 64, 128, 256, 512, 1024])
def test_rows_of_the_stages(lq, hb, dtype):
    rng = np.random.default_rng(hb)
    K = hb * (5 if hb >= 512 else 5 * 1024 // hb // 2 + 1)
    gain = torch.exp(2 * randn(rng, 1, K))
    c = 0.8 + 0.4 * torch.rand(K, generator=torch.Generator().manual_seed(hb)).to(DEV)
    for scales in (None, c):
        x = (randn(rng, 2000, K) * gain).to(dtype)
        got = quant(lq, x, hb=hb, c=scales)
        want = stages(x.float().cpu().numpy(), None if scales is None else scales.cpu().numpy(), hb)
        same(got, want.astype(np.float64))
