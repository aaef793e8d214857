"""Gates whose exponential lies below the normal floats: act(g) stays as accurate as a float there is."""
import numpy as np
import pytest
import torch

from tests.gpu_util import DEV, note
from tests.test_gpu_int8 import U32, gate_error, host64, near_codes, quant

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -150             # half a step of the floats below the normal ones


@pytest.fixture(scope="module")
def lq():
    import bit_matmul_amd
    assert torch.cuda.is_available()
    return bit_matmul_amd


def sigmoid(x):
    return np.exp(x) / (1.0 + np.exp(x))


@pytest.mark.parametrize("first,last", [(-87.3, -87.5), (-87.4, -91.0), (-80.0, -91.0)])
def test_silu_of_gates_that_nearly_shut(lq, first, last):
    """g exp(g) is a normal float down to -91.9 where exp(g) is one only down to -87.3: its relative error
    stays what it is elsewhere."""
    g = torch.linspace(first, last, 61, device=DEV)[None]
    g64 = host64(g)
    v = g64 * sigmoid(g64)
    near_codes(quant(lq, torch.ones_like(g), g, "silu"), v, np.abs(v) * (gate_error("silu", g64) + U32))


def test_gelu_of_gates_that_nearly_shut(lq):
    g = torch.linspace(-10.0, -10.14, 47, device=DEV)[None]
    g64 = host64(g)
    v = g64 * sigmoid(2 * np.sqrt(2 / np.pi) * (g64 + 0.044715 * g64 ** 3))
    near_codes(quant(lq, torch.ones_like(g), g, "gelu"), v, np.abs(v) * (gate_error("gelu", g64) + U32))


def test_sigmoid_below_the_normal_floats(lq):
    """The sigmoid itself is such a float from -87.3 on: off by half a step of those, which a large x shows."""
    g = torch.linspace(-86.0, -100.0, 57, device=DEV)[None]
    x = torch.full_like(g, 1e30)
    x[0, :40] = torch.logspace(26, 30, 40, device=DEV)
    g64, x64 = host64(g), host64(x)
    v = x64 * sigmoid(g64)
    near_codes(quant(lq, x, g, "sigmoid"), v, np.abs(v) * (gate_error("sigmoid", g64) + U32) + 1.01 * HALF * x64)


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_gates_far_apart_in_one_row(lq, act):
    """Shut, nearly shut and open gates next to each other, NaN and infinities in other rows."""
    row = np.linspace(-95.0, 95.0, 700)
    g = torch.from_numpy(np.stack([row, row, row, row[::-1]]).astype(np.float32)).to(DEV)
    g[1, 3], g[2, 9] = float("nan"), float("inf")
    x = torch.ones_like(g)
    note(f"lq_quant_rows gates far apart {act}")
    q, s = quant(lq, x, g, act)
    keep = [0, 3]
    g64 = host64(g)[keep]
    v = sigmoid(np.minimum(g64, 0)) * np.where(g64 > 0, 1 / (1 + np.exp(-np.abs(g64))) / 0.5, 1.0)
    v = v * (g64 if act == "silu" else 1.0)
    near_codes((q[keep], s[keep]), v, np.abs(v) * (gate_error(act, g64) + U32) + 1e-37)
    assert np.isnan(s[1]) and np.all(q[1] == 0)
    assert np.isnan(s[2]) == (act == "silu")
