"""The one-launch form of the 8-bit layer: which calls take it, and the loads ahead of its copies in every
combination (row type, length, rows per workgroup, channel scales with and without the transform)."""
import numpy as np
import pytest
import torch

from oracle import int8_ref as ref
from tests.gpu_util import DEV, note
from tests.test_gpu_int8 import BF, F32, check_product, garbage, host64, make_layer, pad16, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lq():
    import bit_matmul_amd
    assert torch.cuda.is_available()
    return bit_matmul_amd


# (N, K, hb, rows of a workgroup, 0: two launches): one, two and four steps a wavefront, two panels
SIZES = [(50, 1000, 1, 16), (50, 1000, 8, 16), (33000, 520, 1, 32), (8201, 520, 8, 32), (77, 2040, 1, 16),
         (77, 2040, 8, 16), (300, 3600, 1, 16), (300, 3600, 16, 16), (8193, 1024, 1024, 32), (65, 4096, 1024, 16),
         (65, 4104, 8, 0)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("scales", [False, True])
@pytest.mark.parametrize("N,K,hb,rows", SIZES)
def test_scales_and_transform_apart(lq, N, K, hb, rows, scales, dtype):
    """Channel scales without the transform and the transform without scales: the bits of the two launches,
    and the product of codes that the oracle finds within half a step (test_gpu_int8 gives T's error)."""
    rng = np.random.default_rng(N + K + hb)
    c = randn(rng, K).abs() + 0.5 if scales else None
    layer, keep = make_layer(lq, rng, N, K, bias=True, hb=hb, c=c)
    p = lq.lq_int8_linear_plan(layer, 1)
    assert (p["rows"] if p["tokens"] == 1 else 0) == rows
    x = randn(rng, 1, K + 1).to(dtype)[:, 1:]
    ws = garbage(lq.lq_int8_linear_workspace_size(layer, 1, dtype))
    y, y2 = torch.empty(1, N, device=DEV), torch.empty(1, N, device=DEV)
    note(f"lq_int8_linear B=1 N={N} K={K} hb={hb} x={dtype} scales={scales} {p}")
    lq.lq_int8_linear(layer, x, 1, y, ws)
    torch.cuda.synchronize()
    # one launch leaves the workspace alone, two write the rows there
    assert bool(torch.all(ws == 0xA5)) == (rows > 0)
    q = torch.empty(1, pad16(K), dtype=torch.int8, device=DEV)[:, :K]
    s = torch.empty(1, device=DEV)
    lq.lq_quant_rows(x, 1, K, q, s, hb=hb, c=c)
    lq.lq_int8_gemm(layer, q, s, 1, y2, garbage(lq.lq_int8_gemm_workspace_size(layer, 1)))
    torch.cuda.synchronize()
    assert torch.equal(y, y2)
    v = ref.transform(host64(x), hb=hb, c=None if c is None else host64(c))
    c64 = np.ones(K) if c is None else host64(c)
    err = (np.log2(hb) + 2) * 2.0 ** -24 * np.abs(host64(x) * c64).reshape(1, -1, hb).sum(axis=2).max() / np.sqrt(hb)
    codes = q.cpu().numpy().astype(np.int64)
    assert np.all(np.abs(codes - ref.quotients(v)) <= 0.5 + 2 * 127 * err / np.abs(v).max() * 1.01)
    _, w, r, b, _ = keep
    check_product(y, ref.product(codes, host64(s), w.cpu().numpy(), host64(r), host64(b)), b, F32)
