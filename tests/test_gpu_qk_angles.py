"""Cosines and sines of the heads' rotation are rounded once.

A pair (1, 0) comes out as (cos t, sin t) themselves: products by 1 and 0 are exact. Rounded once to fp32
they are off by 2^-24 of themselves; an angle taken in fp64 (formed as pos freq, which is the formula's own
rounding, then turned into turns) is off by 2^-51 of itself, and the sums that make sine and cosine of it by 2^-33."""
import numpy as np
import pytest
import torch

from tests.gpu_util import DEV, note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("base,lo,hi", [(10000.0, 0, 4096), (500000.0, 0, 1 << 20), (10000.0, -(1 << 20), 1 << 20),
                                        (10000.0, 0, 1 << 31)])
def test_cosines_and_sines_are_rounded_once(base, lo, hi, interleaved):
    import bit_matmul_amd as lq
    B, dim = 2000, 128
    g = torch.Generator(DEV).manual_seed(hi % 1009)
    pos = torch.randint(lo, hi, (B,), generator=g, device=DEV)
    pos[:9] = torch.arange(9, device=DEV)
    freq = base ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=DEV) / dim)
    # angles at and around the borders of quarters, too
    freq[-8:] = torch.tensor([np.pi / 4, np.pi / 2, np.pi, 2 * np.pi, np.pi / 8, 3 * np.pi / 4, 1e-9, 0.0],
                             dtype=torch.float64, device=DEV)
    first = torch.arange(dim // 2, device=DEV) * (2 if interleaved else 1)
    second = first + (1 if interleaved else dim // 2)
    x, out = torch.zeros(B, 1, dim, device=DEV), torch.empty(B, 1, dim, device=DEV)
    x[:, :, first] = 1.0
    note(f"lq_qk_norm_rope of (1, 0), base={base} positions {lo} to {hi} interleaved={interleaved}")
    lq.lq_qk_norm_rope(pos, freq, q=x, q_out=out, norm=False, interleaved=interleaved)
    torch.cuda.synchronize()
    angle = pos.cpu().numpy().astype(np.float64)[:, None] * freq.cpu().numpy()
    slack = np.abs(angle) * 2.0 ** -51 + 2.0 ** -33
    for place, want in ((first, np.cos(angle)), (second, np.sin(angle))):
        off = np.abs(out[:, 0, place].double().cpu().numpy() - want)
        tol = (np.abs(want) + slack) * 2.0 ** -24 + slack
        assert np.all(off <= tol), (off / tol).max()
