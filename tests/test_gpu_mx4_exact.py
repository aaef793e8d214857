"""4-bit products and layers of data that fp32 sums exactly (tests/mx4_exact.py): equal to the product, at the
longest rows and with scales from one end to the other."""
import pytest
import torch

from oracle import mx4_ref as ref
from tests.gpu_util import DEV, note
from tests.mx4_exact import pair, product
from tests.test_gpu_mx4 import F32, workspace

pytestmark = pytest.mark.gpu

LONG = 1 << 20


@pytest.fixture(scope="module")
def lq():
    import bit_matmul_amd
    assert torch.cuda.is_available()
    return bit_matmul_amd


def gemm(lq, q, w, y=None):
    B, N = q.rows, w.rows
    codes, scales = w.on(DEV)
    layer = lq.mx4_layer_struct(N, w.K, codes, scales)
    y = torch.full((B + 2, N), 9.0, device=DEV)
    note(f"lq_mx4_gemm exact B={B} N={N} K={w.K} {lq.lq_mx4_gemm_plan(layer, B)}")
    lq.lq_mx4_gemm(layer, *q.on(DEV), B, y[1:B + 1], workspace(lq.lq_mx4_gemm_workspace_size(layer, B)))
    torch.cuda.synchronize()
    assert torch.all(y[0] == 9.0) and torch.all(y[B + 1] == 9.0)
    return y[1:B + 1]


@pytest.mark.parametrize("B,N", [(1, 40), (3, 40), (16, 33), (9, 300), (24, 130), (130, 70), (200, 300)])
def test_longest_products_are_exact(lq, B, N):
    for K in (LONG, LONG - 33):
        q, w = pair(B + K % 7, B, N, K, 3)
        assert torch.equal(gemm(lq, q, w).double(), product(q, w, DEV))


def layer_of(lq, q, w):
    """The whole layer of the values that the rows stand for."""
    codes, scales = w.on(DEV)
    layer = lq.mx4_layer_struct(w.rows, w.K, codes, scales)
    x = torch.from_numpy(ref.decode(ref.unpack(q.packed), q.bytes, q.K)).to(F32).to(DEV)
    y = torch.full((q.rows + 1, w.rows), 9.0, device=DEV)
    note(f"lq_mx4_linear exact B={q.rows} N={w.rows} K={w.K}")
    lq.lq_mx4_linear(layer, x, q.rows, y[:q.rows], workspace(lq.lq_mx4_linear_workspace_size(layer, q.rows, F32)))
    torch.cuda.synchronize()
    assert torch.all(y[q.rows] == 9.0)
    return y[:q.rows]


@pytest.mark.parametrize("B,K", [(1, LONG), (1, LONG - 33), (5, LONG - 33)])
def test_longest_layers_are_exact(lq, B, K):
    q, w = pair(B, B, 50, K, 3, top=True)
    assert torch.equal(layer_of(lq, q, w).double(), product(q, w, DEV))


# a token, few, tiles of every width, split reductions
SIZES = [(1, 512, 8192), (2, 100, 4100), (8, 300, 2048), (16, 500, 1111), (20, 100, 16384), (64, 300, 1024), (100, 600, 2600),
         (300, 600, 777), (600, 1100, 1500)]


@pytest.mark.parametrize("B,N,K", SIZES)
def test_scales_from_end_to_end(lq, B, N, K):
    """Scale bytes 0 to 254 on both sides, whose exponents cancel."""
    q, w = pair(N, B, N, K, 127)
    if K >= 4096:
        assert {0, 254} <= set(w.bytes[0].tolist()) | set(q.bytes[0].tolist())
    assert torch.equal(gemm(lq, q, w).double(), product(q, w, DEV))


@pytest.mark.parametrize("edge", [0, 1, 2, 126, 128, 252, 253, 254])
@pytest.mark.parametrize("B", [1, 7, 40, 200])
def test_scales_at_the_ends(lq, B, edge):
    """One byte for all weights, what is left of 254 for all rows."""
    q, w = pair(edge, B, 130, 700, edge - 127, low=edge - 127)
    assert set(w.bytes.ravel().tolist()) == {edge}
    assert torch.equal(gemm(lq, q, w).double(), product(q, w, DEV))


@pytest.mark.parametrize("B,N,K", [(1, 300, 8192), (1, 200, 1000), (1, 100, 16384), (1, 4200, 12288), (3, 200, 2600), (40, 200, 2600)])
def test_layers_of_values_from_end_to_end(lq, B, N, K):
    """Rows from 2^-128 to 2^127 in blocks of their own, which the layer turns into scale bytes 0 to 252."""
    q, w = pair(K, B, N, K, 127, low=-125, top=True)
    assert torch.equal(layer_of(lq, q, w).double(), product(q, w, DEV))


@pytest.mark.parametrize("low", [100, 20])
@pytest.mark.parametrize("B", [3, 16, 40, 300])
def test_products_past_the_floats(lq, B, low):
    """Scales whose product passes the largest float or falls below the smallest, in a row each: infinities of the
    products' sign; floats below the normal ones (2^-154 times a sum: a rounding of 2^-149 for each 128 products
    and each of at most 4 parts joined) or zeros (2^-234); the other rows keep their sums."""
    q, w = pair(B, B, 70, 640, 0)
    w.packed &= 0x77                                     # no negative weights
    w.packed |= 0x11                                     # and no zeros
    w.values = (ref.GRID[ref.unpack(w.packed) & 7])[:, :640]
    want = product(q, w, DEV)
    q.packed[1] &= 0x77
    q.packed[1] |= 0x11
    q.packed[2] = q.packed[1] | 0x88
    places = ref.scale_places(B, 640)[:, :20]
    q.panels[places[1]], q.panels[places[2]], q.panels[places[0]] = 254, 254, 0
    w.panels[ref.scale_places(70, 640)[:35, :20]] = 254  # 2^127 times 2^127
    w.panels[ref.scale_places(70, 640)[35:, :20]] = low  # 2^-127 times less than 1; 2^127 times that: floats
    y, e = gemm(lq, q, w).double(), low - 127
    assert torch.all(y[1, :35] == float("inf")) and torch.all(y[2, :35] == float("-inf"))
    assert torch.all((y[0, 35:] - want[0, 35:] * 2.0 ** (e - 127)).abs() <= (9 * 2.0 ** -149 if low == 100 else 2.0 ** -200))
    assert torch.equal(y[0, :35], want[0, :35])
    assert torch.equal(y[3:, 35:], want[3:, 35:] * 2.0 ** e)
    big = torch.from_numpy(ref.GRID[ref.unpack(q.packed[1:3]) & 7][:, :640]).to(DEV) @ torch.from_numpy(w.values[35:]).to(DEV).T
    assert torch.equal(y[1:3, 35:], big * torch.tensor([[1.0], [-1.0]], device=DEV, dtype=torch.float64) * 2.0 ** (e + 127))
