"""The microscaled 4-bit rows, their product and the whole 4-bit layer against
the fp64 oracle.

* Scales and codes of rows taken as they are equal the oracle's: the quotient
  by a power of two is exact. With a gate or T the 32-bit value before the
  rounding may be off by its own error, derived at each test.
* Products of two codes and their scales are exact in fp32; a sum of K of them
  is off by at most (K / 32 + 8) roundings, each 2^-23 of the sum of the terms'
  magnitudes (the matrix core adds 128 in one instruction in an order of its
  own, an instruction's sum is rounded into fp32, and the parts of a split
  reduction are added: 2^-23, not 2^-24, so that truncation would pass too).
  row_scale, bias and bf16 add their roundings.
"""
import numpy as np
import pytest
import torch

from oracle import int8_ref, mx4_ref as ref
from tests.gpu_util import DEV, note

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lq():
    import bit_matmul_amd
    assert torch.cuda.is_available()
    return bit_matmul_amd


def width(K):
    return 16 * -(-K // 32)


def host64(t):
    return t.double().cpu().numpy()


def randn(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DEV)


def quant(lq, x, gate=None, act="none", hb=1, c=None, ldq=None, fill=0x55):
    """(codes, scale bytes (rows, blocks)); nothing but what the rows own was written."""
    B, K = x.shape
    ld = width(K) if ldq is None else ldq
    buf = torch.full((B + 2, ld), fill, dtype=torch.uint8, device=DEV)
    n = lq.lq_mx4_scale_size(B, K)
    scale = torch.full((n + 32,), fill, dtype=torch.uint8, device=DEV)
    note(f"lq_mx4_quant_rows B={B} K={K} x={x.dtype} ldx={x.stride(0)} gate={gate is not None} act={act} hb={hb}")
    lq.lq_mx4_quant_rows(x, B, K, buf[1:B + 1], scale[16:16 + n], gate=gate,
                         act=getattr(lq, "LQ_ACT_" + act.upper()), hb=hb, c=c)
    torch.cuda.synchronize()
    b, s = buf.cpu().numpy(), scale.cpu().numpy()
    assert np.all(b[0] == fill) and np.all(b[B + 1:] == fill) and np.all(b[1:B + 1, width(K):] == fill)
    assert np.all(s[:16] == fill) and np.all(s[16 + n:] == fill)
    s = s[16:16 + n]
    places = ref.scale_places(B, K)
    own = np.zeros(n, dtype=bool)
    own[places] = True
    assert np.all(s[~own] == fill)
    nb = -(-K // 32)
    assert np.all(s[places[:, nb:]] == 0)
    code = ref.unpack(b[1:B + 1, :width(K)])
    assert np.all(code[:, K:] == 0)
    return code, s[places[:, :nb]]


def same(got, x64):
    code, scale = ref.quantise(x64)
    assert np.array_equal(got[1], scale), np.argwhere(got[1] != scale)[:4]
    # (the sign of a value that rounds to zero stands for nothing)
    k = x64.shape[1]
    a, b = ref.decode(got[0], got[1], k), ref.decode(code, scale, k)
    assert np.array_equal(a, b, equal_nan=True), np.argwhere(a != b)[:4]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,K", [(1, 1), (3, 7), (2, 31), (2, 32), (3, 33), (17, 256), (1, 257), (2, 512), (2, 1023),
                                 (5, 1025), (7, 4099), (33, 4100), (3, 8192), (1, 28672), (2, 70001), (300, 64)])
def test_quant_rows_are_exact(lq, B, K, dtype):
    rng = np.random.default_rng(K + B)
    x = (randn(rng, B, K) * torch.exp(3 * randn(rng, B, K))).to(dtype)
    same(quant(lq, x), host64(x))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_quant_rows_ties_borders_and_extremes(lq, dtype):
    """Every tie and its neighbours, at scales from the smallest to the largest float, zeros,
    blocks of one value, of subnormals, saturation, infinities and NaN in a block of their own."""
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, 7.0, 7.875]
    vals = np.array([m * s for m in mids for s in (1, -1)] + [4.0, -4.0, 0.5, 6.0, 2.0, 3.0, 1.5, 1.0, 7.5, 0.125, 0.0, -0.0])
    assert len(vals) == 32
    rows = []
    for p in (-149, -140, -127, -126, -125, -124, -20, 0, 30, 124, 125):
        rows.append(np.ldexp(vals, p))
    rows.append(np.zeros(32))
    one = np.zeros(32)
    one[31] = -2.0 ** -149
    rows.append(one)
    rows.append(np.full(32, 3.3895313892515355e38))
    x = torch.tensor(np.stack(rows), dtype=torch.float64).to(dtype)
    near = torch.nextafter(x, torch.full_like(x, float("inf"))) if dtype == F32 else x * (1 + 2.0 ** -7)
    x = torch.cat((x, torch.where(torch.isfinite(near), near, x)), dim=0).to(DEV)
    same(quant(lq, x), host64(x))
    for bad in (float("inf"), float("-inf"), float("nan")):
        y = x.repeat(1, 3)
        y[:, 40] = bad
        code, scale = quant(lq, y)
        assert np.all(scale[:, 1] == 255) and np.all(code[:, 32:64] == 0)
        same((code, scale), host64(y))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_quant_rows_strides(lq, dtype):
    """Rows of a wider tensor at odd element offsets, ld of the codes larger than a row."""
    rng = np.random.default_rng(5)
    wide = randn(rng, 19, 999).to(dtype)
    x = wide[1:18, 3:3 + 901]
    same(quant(lq, x, ldq=512), host64(x))


def value_error(x64, gate64=None, act="none", hb=1, c=None):
    """(v, how far the kernel's fp32 v may be from it): gate and x are exact in fp32; act is good to 8 units
    of 2^-24 (at the gates drawn here), the products by it and by c round once each; a sum of hb values through
    log2 hb stages rounds every partial sum, each at most the sum of the magnitudes; the factor rounds twice."""
    v = int8_ref.transform(x64, gate64, act, hb, c)
    t = x64 if gate64 is None else x64 * int8_ref.act(act, gate64)
    t = np.abs(t if c is None else t * np.asarray(c, dtype=np.float64))
    units = (9 if gate64 is not None else 0) + (1 if c is not None else 0)
    if hb > 1:
        size = t.reshape(t.shape[0], -1, hb).sum(axis=2, keepdims=True) / np.sqrt(hb)
        size = np.broadcast_to(size, (t.shape[0], t.shape[1] // hb, hb)).reshape(t.shape)
        return v, size * ((units + np.log2(hb) + 2) * U32)
    return v, t * (units * U32)


def near_codes(got, v, off):
    """Every scale is that of some maximum within its error, and every code the nearest to some value within its."""
    code, scale = got
    K = v.shape[1]
    b, o = ref.blocks(v), ref.blocks(off)
    top, slack = np.abs(b).max(axis=2), o.max(axis=2)
    low = ref.exponents((np.maximum(top - slack, 0)).repeat(32, axis=1))
    high = ref.exponents((top + slack).repeat(32, axis=1))
    e = scale.astype(int) - 127
    assert np.all((low <= e) & (e <= high))
    step = np.ldexp(1.0, e)[:, :, None]
    d = ref.blocks(ref.decode(code, scale, K)) / step
    a = np.abs(b) / step
    half = np.where(np.abs(d) < 2, 0.25, np.where(np.abs(d) < 4, 0.5, 1.0))        # above d; below it at most that
    sat = (a > 6) & (np.abs(d) == 6)
    assert np.all(sat | (np.abs(d - b / step) <= half + o / step))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("hb", [2, 4, 8, 16, 32, 64, 128, 256, 512, 1024])
def test_quant_rows_transform(lq, hb, dtype):
    rng = np.random.default_rng(hb)
    K = hb * (5 if hb >= 512 else 5 * 1024 // hb // 2 + 1)
    x = randn(rng, 5, K).to(dtype)
    c = 0.8 + 0.4 * torch.rand(K, generator=torch.Generator().manual_seed(hb)).to(DEV)
    got = quant(lq, x, hb=hb, c=c)
    near_codes(got, *value_error(host64(x), hb=hb, c=host64(c)))
    got = quant(lq, x, hb=hb)
    near_codes(got, *value_error(host64(x), hb=hb))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "sigmoid", "tanh"])
@pytest.mark.parametrize("hb", [1, 256])
def test_quant_rows_gate(lq, act, hb, dtype):
    rng = np.random.default_rng(11)
    K = 2048 + 256
    both = randn(rng, 18, 2 * K).to(dtype)
    c = 0.8 + 0.4 * torch.rand(K, generator=torch.Generator().manual_seed(3)).to(DEV)
    gate, up = both[:, :K], both[:, K:]
    got = quant(lq, up, gate=gate, act=act, hb=hb, c=c)
    near_codes(got, *value_error(host64(up), host64(gate), act, hb, host64(c)))




class Layer:
    """A layer's tensors: random codes of every value, scales of a wide range, rows ldw bytes apart; what
    lies past K and past N is garbage."""

    def __init__(self, lq, N, K, seed=0, row_scale=True, bias=False, ldw=None, spread=3, **kw):
        rng = np.random.default_rng(seed)
        nb = -(-K // 32)
        code = rng.integers(0, 16, size=(N, 32 * nb), dtype=np.uint8)
        scale = (127 + rng.integers(-spread, spread + 1, size=(N, nb))).astype(np.uint8)
        self.w64 = ref.decode(code, scale, K)
        ld = width(K) if ldw is None else ldw
        data = rng.integers(0, 256, size=(N, ld), dtype=np.uint8)
        data[:, :width(K)] = ref.pack(code)
        self.w = torch.from_numpy(data).to(DEV)
        self.scale = torch.from_numpy(ref.panels(scale, K, fill=255)).to(DEV)
        self.r = (0.5 + torch.rand(N, generator=torch.Generator().manual_seed(seed))).to(DEV) if row_scale else None
        self.bias = randn(rng, N) if bias else None
        self.N, self.K = N, K
        self.struct = lq.mx4_layer_struct(N, K, self.w, self.scale, self.r, bias=self.bias, **kw)


class Rows:
    """Random 4-bit rows with garbage past K and in the scales of rows and blocks that are none."""

    def __init__(self, B, K, seed=1, ldq=None, spread=3):
        rng = np.random.default_rng(seed)
        nb = -(-K // 32)
        code = rng.integers(0, 16, size=(B, 32 * nb), dtype=np.uint8)
        scale = (127 + rng.integers(-spread, spread + 1, size=(B, nb))).astype(np.uint8)
        self.q64 = ref.decode(code, scale, K)
        ld = width(K) if ldq is None else ldq
        data = rng.integers(0, 256, size=(B, ld), dtype=np.uint8)
        data[:, :width(K)] = ref.pack(code)
        self.q = torch.from_numpy(data).to(DEV)
        self.scale = torch.from_numpy(ref.panels(scale, K, fill=255)).to(DEV)


def h64(t):
    return None if t is None else host64(t)


def workspace(n):
    return torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV) if n else None


def near_product(y, rows64, lay, extra=0.0):
    want, size = ref.product(rows64, lay.w64, h64(lay.r), h64(lay.bias))
    tol = size * ((lay.K / 32 + 8) * 2.0 ** -23) + 3 * U32 * (np.abs(want) + np.abs(0 if lay.bias is None else h64(lay.bias)))
    if y.dtype == BF:
        tol = tol + (np.abs(want) + tol) * U16
    got = host64(y)
    assert np.all(np.abs(got - want) <= tol + extra), (np.abs(got - want) / (tol + 1e-300)).max()


def run_gemm(lq, lay, rows, B, dtype, ldy=None):
    ld = lay.N if ldy is None else ldy
    buf = torch.full((B + 2, ld), -7.0, dtype=dtype, device=DEV)
    y = buf[1:B + 1, :lay.N]
    ws = workspace(lq.lq_mx4_gemm_workspace_size(lay.struct, B))
    note(f"lq_mx4_gemm B={B} N={lay.N} K={lay.K} {dtype} ldy={ld} {lq.lq_mx4_gemm_plan(lay.struct, B)}")
    lq.lq_mx4_gemm(lay.struct, rows.q, rows.scale, B, y, ws)
    torch.cuda.synchronize()
    assert torch.all(buf[0] == -7) and torch.all(buf[B + 1] == -7) and torch.all(buf[:, lay.N:] == -7)
    if ws is not None:
        assert torch.all(ws[:lq.LQ_WS_CONTROL_BYTES] == 0xA5)
    return y


SIZES = [(1, 1, 1), (1, 16, 32), (2, 17, 31), (3, 33, 33), (1, 512, 512), (5, 100, 129), (16, 64, 255), (17, 80, 256),
         (4, 40, 257), (15, 1000, 2050), (31, 130, 385), (33, 300, 1000), (64, 257, 4100), (100, 96, 513), (1, 5125, 4099),
         (8, 333, 28672), (129, 520, 1111), (300, 600, 777), (257, 290, 12345), (700, 515, 640), (513, 1025, 300)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,N,K", SIZES)
def test_gemm(lq, B, N, K, dtype):
    lay = Layer(lq, N, K, seed=N + K, bias=B % 2 == 0, row_scale=B % 3 != 0)
    y = run_gemm(lq, lay, rows := Rows(B, K, seed=B), B, dtype, ldy=N + 3)
    near_product(y, rows.q64, lay)


def test_gemm_row_strides(lq):
    lay = Layer(lq, 75, 1030, ldw=1040, bias=True)
    rows = Rows(37, 1030, ldq=784)
    near_product(run_gemm(lq, lay, rows, 37, F32, ldy=81), rows.q64, lay)


@pytest.mark.parametrize("B,N,K", [(3, 40, 700), (130, 300, 700)])
def test_gemm_scales_from_end_to_end(lq, B, N, K):
    """Scale bytes from 0 to 254 (products far below and above the floats vanish or are infinite; here their
    sums stay among the floats), and NaN scales that spoil their row or column and no other."""
    lay, rows = Layer(lq, N, K, spread=60), Rows(B, K, spread=3)
    near_product(run_gemm(lq, lay, rows, B, F32), rows.q64, lay)
    places = ref.scale_places(max(N, B), K)
    clean = run_gemm(lq, lay, rows, B, F32).clone()
    lay.scale[int(places[5, 21])] = 255
    rows.scale[int(ref.scale_places(B, K)[2, 0])] = 255
    y = run_gemm(lq, lay, rows, B, F32)
    bad = torch.zeros(B, N, dtype=torch.bool, device=DEV)
    bad[2, :] = True
    bad[:, 5] = True
    assert torch.all(torch.isnan(y[bad]))
    assert torch.equal(y[~bad], clean[~bad])


LAYERS = [(1, 512, 512, 512), (1, 300, 100, 1), (1, 96, 8192, 1024), (7, 130, 2048, 256), (16, 64, 4099, 1),
          (65, 200, 1280, 128), (333, 77, 515, 1), (300, 520, 2048, 1024)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,N,K,hb", LAYERS)
def test_linear_is_rows_and_product(lq, B, N, K, hb, dtype):
    """The whole layer gives the codes of lq_mx4_quant_rows through the product."""
    rng = np.random.default_rng(B + K)
    c = (0.8 + 0.4 * torch.rand(K, generator=torch.Generator().manual_seed(3))).to(DEV) if hb > 1 else None
    lay = Layer(lq, N, K, bias=True, hb=hb, c=c)
    for act in (None, "silu"):
        both = randn(rng, B, 2 * K + 1).to(dtype)
        gate, x = (both[:, :K] if act else None), both[:, K:2 * K]
        y = torch.full((B + 1, N), -7.0, dtype=dtype, device=DEV)
        ws = workspace(lq.lq_mx4_linear_workspace_size(lay.struct, B, dtype))
        note(f"lq_mx4_linear B={B} N={N} K={K} hb={hb} {dtype} act={act}")
        how = dict(gate=gate, act=lq.LQ_ACT_SILU) if act else {}
        lq.lq_mx4_linear(lay.struct, x, B, y[:B], ws, **how)
        torch.cuda.synchronize()
        assert torch.all(y[B] == -7) and torch.all(ws[:lq.LQ_WS_CONTROL_BYTES] == 0xA5)
        code, scale = quant(lq, x, gate=gate, act=act or "none", hb=hb, c=c)
        near_product(y[:B], ref.decode(code, scale, K), lay)
