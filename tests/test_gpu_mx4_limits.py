"""The 4-bit rows and products, and the heads' norms and rotation, at their largest sizes: the longest rows, more
rows than one axis of a launch has, the most tokens and heads; heads that a NaN or an infinity spoils."""
import numpy as np
import pytest
import torch

from oracle import mx4_ref as ref
from tests.gpu_util import DEV, note
from tests.test_gpu_mx4 import BF, F32, Layer, Rows, host64, near_codes, near_product, quant, randn, run_gemm, value_error, width, workspace
from tests.test_gpu_qk_norm_rope import check, freqs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lq():
    import bit_matmul_amd
    assert torch.cuda.is_available()
    return bit_matmul_amd


@pytest.mark.parametrize("hb,dtype", [(1, F32), (1024, BF)])
def test_longest_rows(lq, hb, dtype):
    rng = np.random.default_rng(hb)
    K = lq.LQ_MX4_MAX_K
    x, g = randn(rng, 2, K).to(dtype), randn(rng, 2, K).to(dtype)
    c = 0.8 + 0.4 * torch.rand(K, generator=torch.Generator().manual_seed(hb)).to(DEV)
    got = quant(lq, x, gate=g, act="silu", hb=hb, c=c)
    near_codes(got, *value_error(host64(x), host64(g), "silu", hb, host64(c)))


@pytest.mark.parametrize("B,N", [(1, 40), (3, 40), (16, 33), (130, 70)])
def test_longest_products(lq, B, N):
    """Of K values, and of 33 fewer."""
    for K in (lq.LQ_MX4_MAX_K, lq.LQ_MX4_MAX_K - 33):
        lay = Layer(lq, N, K, seed=B, bias=True)
        near_product(run_gemm(lq, lay, rows := Rows(B, K, seed=N), B, F32), rows.q64, lay)


def test_longest_layer(lq):
    """The whole layer of one token, in two launches: the codes of lq_mx4_quant_rows through the product."""
    K, N = lq.LQ_MX4_MAX_K, 50
    lay = Layer(lq, N, K, seed=5)
    x = randn(np.random.default_rng(5), 1, K)
    y = torch.empty(1, N, device=DEV)
    note("lq_mx4_linear of the longest row")
    lq.lq_mx4_linear(lay.struct, x, 1, y, workspace(lq.lq_mx4_linear_workspace_size(lay.struct, 1, F32)))
    torch.cuda.synchronize()
    near_product(y, ref.decode(*ref.quantise(host64(x)), K), lay)


def test_more_rows_than_one_axis(lq):
    """2^22 + 37 rows, copies of 1000: the codes and scales of the 1000."""
    rows, K = (1 << 22) + 37, 40
    base = randn(np.random.default_rng(6), 1000, K).to(BF)
    code, scale = quant(lq, base)
    pick = torch.arange(rows, device=DEV) % 1000
    x = base[pick]
    q = torch.full((rows, width(K)), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((lq.lq_mx4_scale_size(rows, K),), 0x55, dtype=torch.uint8, device=DEV)
    note(f"lq_mx4_quant_rows B={rows}")
    lq.lq_mx4_quant_rows(x, rows, K, q, s)
    torch.cuda.synchronize()
    want = torch.from_numpy(ref.pack(np.pad(code, ((0, 0), (0, 64 - code.shape[1]))))).to(DEV)
    assert torch.equal(q, want[pick])
    row = torch.arange(rows, device=DEV)
    for j in range(2):
        assert torch.equal(s[row // 16 * 128 + 8 * (row % 16) + 2 * j], torch.from_numpy(scale[:, j]).to(DEV)[pick])


@pytest.mark.parametrize("B", [1, 2, 40])
def test_many_outputs(lq, B):
    """1000003 outputs, copies of 1000 rows of weights: the same bits."""
    N, K = 1000003, 64
    few = Layer(lq, 1000, K, row_scale=False)
    pick = torch.arange(N, device=DEV) % 1000
    codes, scales = few.w[pick], torch.full((lq.lq_mx4_scale_size(N, K),), 0, dtype=torch.uint8, device=DEV)
    row, old = torch.arange(N, device=DEV), pick
    for j in range(2):
        scales[row // 16 * 128 + 8 * (row % 16) + 2 * j] = few.scale[old // 16 * 128 + 8 * (old % 16) + 2 * j]
    x = randn(np.random.default_rng(B), B, K)
    layer = lq.mx4_layer_struct(N, K, codes, scales)
    outs = []
    for lay, n in ((few.struct, 1000), (layer, N)):
        y = torch.empty(B, n, device=DEV)
        note(f"lq_mx4_linear B={B} N={n}")
        lq.lq_mx4_linear(lay, x, B, y, workspace(lq.lq_mx4_linear_workspace_size(lay, B, F32)))
        outs.append(y)
    torch.cuda.synchronize()
    # (a block of 64 values is one product: no kernel or split sums it in another order)
    assert torch.equal(outs[1], outs[0][:, pick])


@pytest.mark.parametrize("norm", [False, True])
def test_most_tokens(lq, norm):
    """2^20 tokens: those of the last and first ones as the oracle has them, all of them as calls of a few."""
    B, rng = 1 << 20, np.random.default_rng(7)
    x = randn(rng, B, 1, 6)
    pos, freq = torch.arange(B, device=DEV, dtype=torch.int32), freqs(4)
    out, parts = torch.empty_like(x), torch.empty_like(x)
    note(f"lq_qk_norm_rope B={B}")
    lq.lq_qk_norm_rope(pos, freq, q=x, q_out=out, norm=norm)
    for b in range(0, B, 1 << 17):
        e = b + (1 << 17)
        lq.lq_qk_norm_rope(pos[b:e], freq, k=x[b:e], k_out=parts[b:e], norm=norm)
    torch.cuda.synchronize()
    assert torch.equal(out, parts)
    for at in (slice(0, 999), slice(B - 999, B)):
        check(out[at], x[at], pos[at].cpu().numpy(), freq.cpu().numpy(), None, norm, False, 1e-5, False)


@pytest.mark.parametrize("B,dim,rot", [(2, 4, 4), (1, 24, 20)])
def test_most_heads(lq, B, dim, rot):
    rng = np.random.default_rng(9)
    q, k = randn(rng, B, 1 << 16, dim), randn(rng, B, 1 << 16, dim)
    pos, freq, w = torch.tensor([77, -3][:B], device=DEV), freqs(rot), 1 + 0.2 * randn(rng, dim)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    note(f"lq_qk_norm_rope of 65536 heads, dim {dim}")
    lq.lq_qk_norm_rope(pos, freq, q=q, k=k, q_out=qo, k_out=ko, w_k=w)
    torch.cuda.synchronize()
    p, f = pos.cpu().numpy(), freq.cpu().numpy()
    check(qo, q, p, f, None, True, False, 1e-5, False)
    check(ko, k, p, f, w, True, False, 1e-5, False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_spoilt_heads_spoil_no_others(lq, interleaved):
    """Normed heads that hold a NaN or an infinity have it in every output that it reaches; the others keep their bits,
    and so do those of a head whose squares pass the largest float."""
    rng = np.random.default_rng(10)
    x = randn(rng, 4, 9, 80)
    x[1, 3] *= 1e25
    pos, freq = torch.tensor([0, 5, 1 << 20, 9], device=DEV), freqs(60)
    clean, out = torch.empty_like(x), torch.empty_like(x)
    lq.lq_qk_norm_rope(pos, freq, q=x, q_out=clean, interleaved=interleaved)
    torch.cuda.synchronize()
    check(clean, x, pos.cpu().numpy(), freq.cpu().numpy(), None, True, False, 1e-5, interleaved)
    x[0, 0, 3], x[1, 4, 79], x[3, 8, 41] = float("nan"), float("inf"), float("-inf")
    note("lq_qk_norm_rope with NaN and infinities")
    lq.lq_qk_norm_rope(pos, freq, q=x, q_out=out, interleaved=interleaved)
    torch.cuda.synchronize()
    bad = torch.zeros(4, 9, dtype=torch.bool, device=DEV)
    bad[0, 0] = bad[1, 4] = bad[3, 8] = True
    assert torch.equal(out[~bad], clean[~bad])
    assert torch.isnan(out[0, 0]).all()
    # (an infinite head: x / inf, and inf / inf where it is infinite)
    assert torch.isnan(out[1, 4, 79]) and torch.all(out[1, 4, :79] == 0)
    assert torch.isnan(out[3, 8]).sum() == 2
