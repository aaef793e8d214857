"""Refusals of lq_qk_norm_rope's positions and frequencies."""
import pytest
import torch

from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


def test_positions_and_frequencies_that_are_none():
    import bit_matmul_amd as lq
    x, out = torch.ones(3, 2, 32, device=DEV), torch.zeros(3, 2, 32, device=DEV)
    pos, freq = torch.arange(3, device=DEV), torch.rand(16, dtype=torch.float64, device=DEV)
    with pytest.raises(ValueError, match="pos must be int32 or int64"):
        lq.lq_qk_norm_rope(None, freq, q=x, q_out=out)
    with pytest.raises(ValueError, match="pos must be int32 or int64"):
        lq.lq_qk_norm_rope([0, 1, 2], freq, q=x, q_out=out)
    with pytest.raises(ValueError, match="freq must be a float64 tensor"):
        lq.lq_qk_norm_rope(pos, [0.5] * 16, q=x, q_out=out)
    torch.cuda.synchronize()
    assert torch.all(out == 0)
    lq.lq_qk_norm_rope(None, freq[:0], q=x, q_out=out)         # nothing is rotated: no positions are needed
    torch.cuda.synchronize()
    assert torch.all(out != 0)
