"""The 4-bit layer of one token on both sides of the rule that takes one launch or two: the product of
lq_mx4_quant_rows' rows, with rows in the workspace or without."""
import numpy as np
import pytest
import torch

from oracle import mx4_ref as ref
from tests.gpu_util import DEV, note
from tests.test_gpu_mx4 import BF, F32, Layer, near_product, quant, randn, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lq():
    import bit_matmul_amd
    assert torch.cuda.is_available()
    return bit_matmul_amd


@pytest.mark.parametrize("N,K,hb,act,dtype,one", [
    (28672, 5120, 1024, None, BF, False), (28672, 5120, 1, None, BF, True), (28672, 5120, 1, "silu", F32, False),
    (40000, 1024, 1024, "silu", BF, False), (40000, 1024, 1024, None, BF, True), (131072, 512, 1, "gelu", F32, False),
    (28672, 2560, 512, "silu", BF, False), (9000, 8192, 1024, "silu", BF, True), (28672, 8192, 1024, None, F32, True),
    (300, 12288, 1024, "silu", BF, False), (300, 12288, 1024, None, F32, True), (300, 14336, 1024, "silu", F32, True),
    (500, 9000, 8, None, BF, True), (4096, 10240, 1, "gelu", BF, True), (4097, 10240, 1, None, BF, False),
    (9000, 16384, 1, None, F32, True), (9000, 16384, 1024, None, BF, False), (33, 16376, 8, None, F32, True)])
def test_one_launch_or_two(lq, N, K, hb, act, dtype, one):
    rng = np.random.default_rng(N + K)
    c = (0.8 + 0.4 * torch.rand(K, generator=torch.Generator().manual_seed(3))).to(DEV) if hb > 1 else None
    lay = Layer(lq, N, K, bias=True, hb=hb, c=c)
    x, g = randn(rng, 1, K).to(dtype), randn(rng, 1, K).to(dtype) if act else None
    y = torch.full((2, N), 4.0, dtype=dtype, device=DEV)
    ws = workspace(lq.lq_mx4_linear_workspace_size(lay.struct, 1, dtype))
    how = dict(gate=g, act=getattr(lq, "LQ_ACT_" + act.upper())) if act else {}
    note(f"lq_mx4_linear one token N={N} K={K} hb={hb} {dtype} act={act}")
    lq.lq_mx4_linear(lay.struct, x, 1, y, ws, **how)
    torch.cuda.synchronize()
    if torch.cuda.get_device_properties(0).multi_processor_count == 256:
        assert bool(torch.all(ws == 0xA5)) == one
    assert torch.all(ws[:lq.LQ_WS_CONTROL_BYTES] == 0xA5) and torch.all(y[1] == 4.0)
    code, scale = quant(lq, x, gate=g, act=act or "none", hb=hb, c=c)
    near_product(y[:1], ref.decode(code, scale, K), lay)
