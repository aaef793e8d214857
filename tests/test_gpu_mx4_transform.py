"""T of 4-bit rows rounds a result once, whatever hb.

Whole numbers below 2^24 / hb have sums that fp32 holds exactly, so a value of T x is such a sum S times
1 / sqrt(hb): a power of two and, for an odd log2 hb, sqrt(2). The product by it rounds once (2^-24 of the
value), and sqrt(2) as a float is off by 2^-25.79 of itself: v is off by 1.29 x 2^-24 of itself, however
large the values are that made S. Scales and codes have to be those of such a v."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_util import DEV, note
from tests.test_gpu_mx4 import F32, width

pytestmark = pytest.mark.gpu

ROWS, K = 4096, 4096


@pytest.fixture(scope="module")
def lq():
    import bit_matmul_amd
    assert torch.cuda.is_available()
    return bit_matmul_amd


def sums(x, hb):
    """The unnormalised transform of whole numbers, exact in 64 bits."""
    v = x.double()
    h = 1
    while h < hb:
        v = v.reshape(ROWS, -1, 2, h)
        v = torch.stack((v[:, :, 0] + v[:, :, 1], v[:, :, 0] - v[:, :, 1]), dim=2)
        h *= 2
    return v.reshape(ROWS, K)


@pytest.mark.parametrize("hb", [2, 4, 8, 32, 128, 256, 512, 1024])
def test_a_result_is_rounded_once(lq, hb):
    g = torch.Generator(DEV).manual_seed(hb)
    most = (1 << 24) // hb
    q = torch.empty(ROWS, width(K), dtype=torch.uint8, device=DEV)
    scale = torch.empty(lq.lq_mx4_scale_size(ROWS, K), dtype=torch.uint8, device=DEV)
    row, block = torch.arange(ROWS, device=DEV)[:, None], torch.arange(K // 32, device=DEV)
    unit, inside = block // 8, block % 8
    places = (row // 16) * (128 * (K // 256)) + 128 * unit + 8 * (row % 16) + 2 * (inside % 4) + inside // 4
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=DEV)
    rounding = (1.29 if math.log2(hb) % 2 else 0.0) * 2.0 ** -24        # (by a power of two: exact)
    for turn in range(4):
        x = torch.randint(-most + 1, most, (ROWS, K), generator=g, device=DEV).to(F32)
        note(f"lq_mx4_quant_rows of whole numbers, hb={hb}, {turn}")
        lq.lq_mx4_quant_rows(x, ROWS, K, q, scale, hb=hb)
        v = sums(x, hb) / math.sqrt(hb)
        a, off = v.abs(), v.abs() * rounding
        e = scale[places].int() - 127
        top = a.reshape(ROWS, -1, 32).amax(dim=2)
        low, high = (torch.frexp(top * f).exponent - 3 for f in (1 - rounding, 1 + rounding))
        assert torch.all((low <= e) & (e <= high))
        step = ((e.long() + 1023) << 52).view(torch.float64)[:, :, None]        # 2^e, exactly
        code = torch.stack((q & 15, q >> 4), dim=2).reshape(ROWS, -1, 32)
        d, sign = grid[(code & 7).long()], torch.where(code > 7, -1.0, 1.0)
        u, o = (v.reshape(code.shape) / step) * sign, off.reshape(code.shape) / step
        # halfway to the next value up, and down; a tie belongs to the even code, which either bound lets pass
        up = torch.where(d < 2, 0.25, torch.where(d < 4, 0.5, torch.where(d < 6, 1.0, np.inf)))
        down = torch.where(d <= 2, 0.25, torch.where(d <= 4, 0.5, 1.0))
        bad = (u > d + up + o) | (u < d - down - o)
        wrong = int(bad.sum())
        assert wrong == 0, (v.reshape(code.shape)[bad][:4], d[bad][:4])
