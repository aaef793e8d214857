"""The sign of zeros in 4-bit rows."""
import pytest
import torch

from tests.gpu_util import DEV, note
from tests.test_gpu_mx4 import quant

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_zeros_keep_their_sign(dtype):
    import bit_matmul_amd as lq
    x = torch.zeros(1, 96, device=DEV)
    x[0, :32] = -0.0
    x[0, 32], x[0, 40], x[0, 41] = 4.0, -0.2, 0.2               # 0.2 of a step of 0.5: zero
    note(f"lq_mx4_quant_rows of zeros {dtype}")
    code, scale = quant(lq, x.to(dtype))
    assert scale.tolist() == [[0, 127, 0]]
    assert code[0, :32].tolist() == [8] * 32 and code[0, 64:].tolist() == [0] * 32
    assert code[0, 32:64].tolist() == [6] + [0] * 7 + [8] + [0] * 23
