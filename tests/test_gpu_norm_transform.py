"""The norms in front of an 8-bit layer that carries T: the norm's 8-bit rows hold no T, so its values go
through the layer's own rows."""
import numpy as np
import pytest
import torch

from oracle import int8_ref as ref
from tests.gpu_util import DEV, note
from tests.test_gpu_int8 import BF, F32, U32, check_product, garbage, host64, make_layer, near_codes, randn, rows8
from tests.test_gpu_norm_block import norm_err

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lq():
    import bit_matmul_amd
    assert torch.cuda.is_available()
    return bit_matmul_amd


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B", [1, 30, 130])
@pytest.mark.parametrize("K,hb", [(2048, 1024), (5120, 512), (1000, 8)])
def test_norm_values_into_a_layer_with_the_transform(lq, B, K, hb, dtype):
    """lq_norm_block's values through lq_int8_linear: the bits of lq_quant_rows with the layer's hb and c and
    lq_int8_gemm, whose codes lie within half a step and T's error of T of those values."""
    rng = np.random.default_rng(B + K)
    N = 200
    c, w = randn(rng, K).abs() + 0.5, randn(rng, K)
    layer, keep = make_layer(lq, rng, N, K, bias=True, hb=hb, c=c)
    h, a = randn(rng, B, K).to(dtype), torch.empty(B, K, dtype=dtype, device=DEV)
    y, y2 = torch.empty(B, N, device=DEV), torch.empty(B, N, device=DEV)
    note(f"lq_norm_block into a layer with T B={B} K={K} hb={hb} {dtype}")
    lq.lq_norm_block(B, K, h=h, pre=True, w_pre=w, a=a)
    lq.lq_int8_linear(layer, a, B, y, garbage(lq.lq_int8_linear_workspace_size(layer, B, dtype)))
    q, s = rows8(B, K)[0], torch.empty(B, device=DEV)
    lq.lq_quant_rows(a, B, K, q, s, hb=hb, c=c)
    lq.lq_int8_gemm(layer, q, s, B, y2, garbage(lq.lq_int8_gemm_workspace_size(layer, B)))
    torch.cuda.synchronize()
    assert torch.equal(y, y2)
    a64, c64 = host64(a), host64(c)
    tot = np.abs(a64 * c64).reshape(B, -1, hb).sum(axis=2, keepdims=True) / np.sqrt(hb)
    err = np.broadcast_to((np.log2(hb) + 2) * U32 * tot, (B, K // hb, hb)).reshape(B, K)
    codes = q.cpu().numpy().astype(np.int64)
    near_codes((codes, s.cpu().numpy()), ref.transform(a64, hb=hb, c=c64), err)
    check_product(y, ref.product(codes, host64(s), keep[1].cpu().numpy(), host64(keep[2]), host64(keep[3])), keep[3], F32)


@pytest.mark.parametrize("B", [1, 40])
def test_channel_scales_in_the_norms_weights(lq, B):
    """Channel scales alone go into w_pre: the norm's 8-bit rows are then those of c a, within the norm's error
    and the roundings of w_pre c and of the product."""
    rng = np.random.default_rng(B)
    N, K = 120, 1500
    c, w = randn(rng, K).abs() + 0.5, randn(rng, K)
    layer, keep = make_layer(lq, rng, N, K, bias=True, c=c)
    h = randn(rng, B, K)
    q, s, y = rows8(B, K)[0], torch.empty(B, device=DEV), torch.empty(B, N, device=DEV)
    note(f"lq_norm_block with channel scales B={B}")
    lq.lq_norm_block(B, K, h=h, pre=True, w_pre=w * c, q=q, scale=s)
    lq.lq_int8_gemm(layer, q, s, B, y, garbage(lq.lq_int8_gemm_workspace_size(layer, B)))
    torch.cuda.synchronize()
    v = ref.rms_norm(host64(h), host64(w), False, float(np.float32(1e-5))) * host64(c)
    codes = q.cpu().numpy().astype(np.int64)
    near_codes((codes, s.cpu().numpy()), v, np.abs(v) * (norm_err(K) + 2 * U32))
    check_product(y, ref.product(codes, host64(s), keep[1].cpu().numpy(), host64(keep[2]), host64(keep[3])), keep[3], F32)
