"""The 8-bit rows, the 8-bit product and the whole 8-bit layer against the
fp64 oracle.

* Codes of rows taken as they are (no gate, no T) equal the oracle's, and so
  do their scales: the kernel decides every rounding as the exact quotient
  does, ties included. With a gate or T the 32-bit value before the rounding
  may be off by its own error, derived at each test: the code then lies within
  half a step and that error of the exact quotient.
* Sums of byte products are exact, so an output is off by its own roundings
  only: the sum to fp32, the product of the scales, their product, the bias
  (each eps / 2 = 2^-24 of a value at most |y| + |bias|), and bf16's 2^-8.
"""
import numpy as np
import pytest
import torch

from oracle import int8_ref as ref
from tests.gpu_util import DEV, note

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lq():
    import bit_matmul_amd
    assert torch.cuda.is_available()
    return bit_matmul_amd


def pad16(K):
    return -(-K // 16) * 16


def rows8(B, K, ld=None, fill=0x55):
    """B int8 rows of K inside a larger buffer of `fill` bytes: (view, buffer)."""
    ld = pad16(K) if ld is None else ld
    buf = torch.full((B + 2, ld), fill, dtype=torch.int8, device=DEV)
    return buf[1:B + 1, :K], buf


def untouched(buf, B, K, fill=0x55):
    """Nothing outside rows 1..B, columns below K rounded up to 16, was written; the pad is zero."""
    b = buf.cpu().numpy()
    assert np.all(b[0] == fill) and np.all(b[B + 1:] == fill)
    assert np.all(b[1:B + 1, pad16(K):] == fill)
    assert np.all(b[1:B + 1, K:pad16(K)] == 0)


def host64(t):
    return t.double().cpu().numpy()


def randn(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DEV)


def quant(lq, x, gate=None, act="none", hb=1, c=None, ldq=None):
    B, K = x.shape
    q, buf = rows8(B, K, ldq)
    scale = torch.full((B + 2,), 7.0, dtype=F32, device=DEV)
    note(f"lq_quant_rows B={B} K={K} x={x.dtype} ldx={x.stride(0)} gate={gate is not None} act={act} hb={hb}")
    lq.lq_quant_rows(x, B, K, q, scale[1:B + 1], gate=gate, act=getattr(lq, "LQ_ACT_" + act.upper()),
                     hb=hb, c=c)
    torch.cuda.synchronize()
    untouched(buf, B, K)
    s = scale.cpu().numpy()
    assert s[0] == 7.0 and s[-1] == 7.0
    return q.cpu().numpy().astype(np.int64), s[1:B + 1]


def same_codes(got, x64):
    q, s = got
    want, _ = ref.codes(x64)
    assert np.array_equal(q, want), np.argwhere(q != want)[:4]
    assert np.array_equal(s, np.abs(x64).max(axis=1).astype(np.float32) / np.float32(127))


# every wavefront count and register shape: one block, a partial one, 16 blocks, 2 and 4 per wavefront
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,K", [(1, 1), (3, 7), (2, 15), (2, 16), (3, 17), (1, 512), (2, 1023), (5, 1025),
                                 (7, 4099), (3, 8192), (2, 16384), (2, 16385), (1, 28672), (2, 32769),
                                 (1, 65536), (300, 64)])
def test_quant_rows_are_exact(lq, B, K, dtype):
    rng = np.random.default_rng(K + B)
    x = (randn(rng, B, K) * torch.exp(randn(rng, B, 1))).to(dtype)
    same_codes(quant(lq, x), host64(x))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_quant_rows_ties_and_extremes(lq, dtype):
    """Quotients that are exact ties (top 127: k + 1/2), rows of zeros, of the smallest and the
    largest values, a row of one sign, the maximum in the last column."""
    K = 261
    rows = []
    half = np.arange(K) * 0.5 - 65.0          # -65 .. 65 in halves, all bf16 values
    half[-1] = 127.0
    rows.append(half)
    rows.append(-half)
    rows.append(half * 2.0 ** -130)           # subnormal
    rows.append(half * 2.0 ** 120)            # near the largest float
    rows.append(np.zeros(K))
    one = np.zeros(K)
    one[3] = -2.0 ** -126
    rows.append(one)
    alt = np.where(np.arange(K) % 2 == 0, 1.0, -1.0)
    rows.append(alt)
    x = torch.tensor(np.stack(rows), dtype=torch.float64).to(dtype).to(DEV)
    q, s = quant(lq, x)
    x64 = host64(x)
    same_codes((q, s), x64)
    assert np.all(q[4] == 0) and s[4] == 0.0
    assert q[0, 0] == -65 and q[0, 1] == -64 and q[0, 131] == 0      # -64.5 -> -64, 0.5 -> 0


def test_quant_rows_near_ties_fp32(lq):
    """Values one and two units of the last place from every half step."""
    K = 1024
    rng = np.random.default_rng(11)
    x = np.zeros((8, K), dtype=np.float32)
    for b in range(8):
        top = np.float32(rng.uniform(0.5, 2.0))
        h = (rng.integers(-126, 126, K) + 0.5) * np.float64(top) / 127.0
        f = h.astype(np.float32)
        step = rng.integers(-2, 3, K, dtype=np.int32)
        x[b] = (f.view(np.int32) + step).view(np.float32)
        x[b, 5] = top
    same_codes(quant(lq, torch.from_numpy(x).to(DEV)), x.astype(np.float64))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_quant_rows_non_finite(lq, dtype):
    rng = np.random.default_rng(3)
    x = randn(rng, 4, 700).to(dtype)
    x[1, 699] = float("nan")
    x[2, 0] = float("-inf")
    q, s = quant(lq, x)
    assert np.isnan(s[1]) and np.isnan(s[2]) and np.all(q[1:3] == 0)
    keep = [0, 3]
    same_codes((q[keep], s[keep]), host64(x)[keep])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_quant_rows_of_slices(lq, dtype):
    """Rows of a wider tensor, from an odd column, into rows further apart."""
    rng = np.random.default_rng(4)
    wide = randn(rng, 9, 3001).to(dtype)
    x = wide[:, 1001:1001 + 1501]
    same_codes(quant(lq, x, ldq=2048), host64(x))


# (gate, act): the gate's 32-bit error. Sigmoid: the exponent's product is carried to 2^-40 or so, exp2 and
# the reciprocal are within one unit each, and 1 + e, the last fused step and the products round: 8 units
# (2^-23) are more than all of them. tanh: the library's 2 units. gelu: its argument (about 3 roundings
# of |2u|) adds 3 * 2^-24 |2u|.
def gate_error(act, g64):
    if act == "none":
        return 2 * U32
    e = 8 * 2 * U32
    if act == "gelu":
        e = e + 4 * U32 * np.abs(1.6 * (g64 + 0.044715 * g64 ** 3))
    return e


def near_codes(got, v64, err):
    """Codes within half a step and `err` (absolute, of v) of the exact quotient."""
    q, s = got
    top = np.abs(v64).max(axis=1, keepdims=True)
    etop = np.max(err, axis=1, keepdims=True)
    slack = 127.0 * (err / top + etop / top) * (1 + 1e-3)
    d = np.abs(q - ref.quotients(v64))
    assert np.all(d <= 0.5 + slack), (d.max(), slack.max())
    assert slack.max() < 0.25                  # (so a wrong code would be seen)
    assert np.all(np.abs(s - top[:, 0] / 127) <= (U32 * top[:, 0] + etop[:, 0]) / 127 * (1 + 1e-3))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("B,K", [(1, 5), (4, 1501), (2, 17000), (1, 40000)])
def test_quant_rows_with_a_gate(lq, B, K, act, dtype):
    rng = np.random.default_rng(K)
    wide = randn(rng, B, 2 * K).to(dtype)
    gate, x = wide[:, :K], wide[:, K:]
    v = ref.transform(host64(x), host64(gate), act)
    err = (np.abs(v) + 1e-30) * (gate_error(act, host64(gate)) + U32)
    near_codes(quant(lq, x, gate, act), v, err)


def test_gate_far_out(lq):
    """Gates where the exponential overflows or vanishes."""
    g = torch.tensor([[-1e30, -200.0, -90.0, -30.0, -1e-30, 0.0, 1e-30, 30.0, 90.0, 200.0, 1e30, 1.0]] * 2,
                     device=DEV)
    x = torch.ones_like(g)
    x[:, 10] = 1e-28
    for act in ("silu", "sigmoid", "tanh"):
        v = ref.transform(host64(x), host64(g), act)
        near_codes(quant(lq, x, g, act), v, np.abs(v) * 20 * U32 + 1e-30)
    g[:, 0], g[:, 10] = -1e10, 1e10           # (the cube of 1e30 overflows to its limits: 0 and g)
    v = ref.transform(host64(x), host64(g), "gelu")
    near_codes(quant(lq, x, g, "gelu"), v, np.abs(v) * 20 * U32 + 1e-20)


@pytest.mark.parametrize("act,size", [("silu", 1.0), ("silu", 3e36), ("gelu", 1.0), ("gelu", 3e36), ("sigmoid", 1e38)])
def test_gate_far_below(lq, act, size):
    """Gates that shut: act(g) x vanishes next to the row's largest value however large g or x are, and keeps
    its relative accuracy while it is a normal float."""
    g = torch.tensor([[-3e38, -1e38, -1e36, -1e30, -1e20, -1e9, -1e3, -150.0, -130.0, -20.0]], device=DEV)
    x = torch.full_like(g, size)
    x[0, 9] = 1.0
    g64 = host64(g)
    # (e^-130 times 1e38 or 130 3e36 is below 1e-17; the largest value is 2e-9 or more)
    err = (gate_error(act, np.maximum(g64, -200.0)) + U32) * np.abs(ref.transform(host64(x), g64, act)) + 1e-17
    if act == "gelu":
        g[0, 9] = 1.0
        g64 = host64(g)
        err = np.full(g64.shape, 1e-6)
    near_codes(quant(lq, x, g, act), ref.transform(host64(x), g64, act), err)
    # a whole row of shut gates: e^-86 is a normal float
    if act != "gelu":
        g = torch.linspace(-80.0, -86.0, 40, device=DEV)[None]
        v = ref.transform(np.ones((1, 40)), host64(g), act)
        near_codes(quant(lq, torch.ones_like(g), g, act), v, np.abs(v) * (gate_error(act, host64(g)) + U32))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("hb", [1, 2, 4, 8, 16, 32, 64, 128, 256, 512, 1024])
@pytest.mark.parametrize("B,blocks", [(2, 1), (1, 17)])
def test_quant_rows_with_the_transform(lq, B, blocks, hb, dtype):
    """T's error: the scale, log2(hb) additions and the final factor each round a partial sum that is
    at most the block's sum of |c x|, so it is at most (log2 hb + 2) 2^-24 of that sum over sqrt(hb)."""
    K = 1024 * blocks if hb > 1 else 1000
    rng = np.random.default_rng(hb)
    x = randn(rng, B, K).to(dtype)
    c = randn(rng, K).abs() + 0.5
    c64 = host64(c)
    v = ref.transform(host64(x), hb=hb, c=c64)
    tot = np.abs(host64(x) * c64).reshape(B, -1, hb).sum(axis=2, keepdims=True) / np.sqrt(hb)
    err = np.broadcast_to((np.log2(hb) + 2) * U32 * tot, (B, K // hb, hb)).reshape(B, K)
    near_codes(quant(lq, x, hb=hb, c=c), v, err)


def test_quant_rows_gate_then_transform(lq):
    rng = np.random.default_rng(8)
    B, K, hb = 2, 2048, 256
    x, g, c = randn(rng, B, K), randn(rng, B, K), randn(rng, K)
    u = ref.transform(host64(x), host64(g), "silu")
    v = ref.transform(u, hb=hb, c=host64(c))
    tot = np.abs(u * host64(c)).reshape(B, -1, hb).sum(axis=2, keepdims=True) / np.sqrt(hb)
    err = np.broadcast_to((8 + 2 + 18) * U32 * tot, (B, K // hb, hb)).reshape(B, K)
    near_codes(quant(lq, x, g, "silu", hb, c), v, err)


# ------------------------------------------------------------------ the product

def make_layer(lq, rng, N, K, bias=False, ldw=None, extreme=False, **kw):
    """(layer, tensors to keep): random weights whose pad bytes hold garbage."""
    buf = torch.from_numpy(rng.integers(-128, 128, (N, ldw or pad16(K)), dtype=np.int8)).to(DEV)
    w = buf[:, :K]
    if extreme:
        w.fill_(-128)
    r = randn(rng, N).abs() * 1e-3 + 1e-4
    b = randn(rng, N) if bias else None
    return lq.int8_layer_struct(N, K, w, r, bias=b, **kw), (buf, w, r, b, kw)


def make_q(rng, B, K, ldq=None):
    """Random codes in rows whose pad bytes hold garbage."""
    buf = torch.full((B, ldq or pad16(K)), 0x77, dtype=torch.int8, device=DEV)
    buf[:, :K] = torch.from_numpy(rng.integers(-128, 128, (B, K), dtype=np.int8)).to(DEV)
    return buf[:, :K]


def garbage(n):
    return torch.full((max(n, 16),), 0xA5, dtype=torch.uint8, device=DEV)


def check_product(y, want, bias, dtype):
    b = 0.0 if bias is None else np.abs(host64(bias))
    tol = 5 * U32 * (np.abs(want) + 2 * b)
    if dtype == BF:
        tol = tol + U16 * (np.abs(want) + tol)
    d = np.abs(host64(y) - want)
    assert np.all(d <= tol), (d.max(), np.argwhere(d > tol)[:4])


def run_gemm(lq, layer, keep, q, scale, dtype, ldy=None):
    B, N = q.shape[0], layer.N
    buf = torch.full((B + 2, ldy or N), 9.0, dtype=dtype, device=DEV)
    y = buf[1:B + 1, :N]
    n = lq.lq_int8_gemm_workspace_size(layer, B)
    ws = garbage(n) if n else None
    note(f"lq_int8_gemm B={B} N={N} K={layer.K} y={dtype} ldq={q.stride(0)} ldw={layer.ldw} ldy={buf.stride(0)}")
    lq.lq_int8_gemm(layer, q, scale, B, y, ws)
    torch.cuda.synchronize()
    assert torch.all(buf[0] == 9.0) and torch.all(buf[B + 1:] == 9.0) and torch.all(buf[:, N:] == 9.0)
    _, w, r, b, _ = keep
    want = ref.product(q.cpu().numpy(), host64(scale), w.cpu().numpy(), host64(r),
                       None if b is None else host64(b))
    check_product(y, want, b, dtype)
    return y


SHAPES = [(1, 1, 1), (1, 16, 16), (2, 15, 63), (3, 17, 64), (15, 33, 65), (16, 31, 127), (17, 100, 128),
          (1, 512, 512), (5, 64, 4099), (33, 257, 300), (64, 129, 1000), (65, 65, 129), (100, 300, 255),
          (127, 128, 256), (128, 255, 257), (129, 513, 640), (200, 77, 2000), (257, 259, 1025), (300, 16, 5000),
          (512, 256, 4096), (600, 700, 900)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,N,K", SHAPES)
def test_int8_gemm(lq, B, N, K, dtype):
    rng = np.random.default_rng(B * 7 + N * 3 + K)
    layer, keep = make_layer(lq, rng, N, K, bias=(B + N) % 2 == 0)
    q = make_q(rng, B, K)
    scale = randn(rng, B).abs() + 0.01
    run_gemm(lq, layer, keep, q, scale, dtype)


@pytest.mark.parametrize("B", [1, 20, 70, 300])
def test_int8_gemm_strided(lq, B):
    rng = np.random.default_rng(B)
    layer, keep = make_layer(lq, rng, 515, 777, bias=True, ldw=1024)
    q = make_q(rng, B, 777, ldq=832)
    scale = randn(rng, B).abs()
    for dtype, ldy in ((F32, 517), (BF, 600), (BF, 517)):
        run_gemm(lq, layer, keep, q, scale, dtype, ldy)


@pytest.mark.parametrize("B", [1, 40, 130])
def test_int8_gemm_largest_sum(lq, B):
    """-128 times -128 over the longest reduction: the largest sum 32 bits have to hold."""
    K = lq.LQ_INT8_MAX_K
    rng = np.random.default_rng(1)
    layer, keep = make_layer(lq, rng, 40, K, extreme=True)
    q = make_q(rng, B, K)
    q.fill_(-128)
    y = run_gemm(lq, layer, keep, q, torch.ones(B, device=DEV), F32)
    assert torch.all(y > 0)


@pytest.mark.parametrize("B", [1, 7, 16])
def test_int8_gemm_largest_sum_of_few_tokens(lq, B):
    """The same with enough rows that the reduction is not split: four wavefronts' parts of it meet."""
    N, K = 8192, lq.LQ_INT8_MAX_K
    w = torch.full((N, pad16(K)), -128, dtype=torch.int8, device=DEV)
    w[N - 1] = 127
    q = torch.full((B, pad16(K)), -128, dtype=torch.int8, device=DEV)
    one = torch.ones(N, device=DEV)
    layer = lq.int8_layer_struct(N, K, w[:, :K], one)
    assert lq.lq_int8_gemm_plan(layer, B)["tokens"] <= 16
    y = torch.zeros(B, N, device=DEV)
    note(f"lq_int8_gemm largest sum B={B} N={N}")
    lq.lq_int8_gemm(layer, q[:, :K], one[:B], B, y, garbage(lq.lq_int8_gemm_workspace_size(layer, B)))
    torch.cuda.synchronize()
    assert torch.all(y[:, :N - 1] == float(np.float32(K * 128 * 128)))
    assert torch.all(y[:, N - 1] == float(np.float32(-K * 128 * 127)))


# (B, N, K, rows and tokens of the tile, whether the reduction is split)
VARIANTS = [
    (20, 16, 700, 32, 32, False), (20, 17, 6000, 32, 32, True), (17, 20001, 48, 64, 32, False),
    (33, 1001, 20001, 64, 32, True), (3, 16, 700, 16, 4, False), (4, 1001, 6001, 16, 4, False),
    (2, 500, 300, 16, 4, False), (5, 3001, 5000, 16, 8, False), (8, 100, 1030, 16, 8, False),
    (9, 2001, 3001, 16, 16, False), (16, 33, 2047, 16, 16, False), (16, 8185, 12001, 32, 16, False),
    (13, 8001, 27000, 32, 16, False), (2, 256, 30001, 32, 32, True), (129, 10001, 48, 64, 64, False),
    (33, 2000, 12001, 128, 64, True),
    (100, 14000, 700, 64, 128, False), (1100, 100, 12001, 64, 128, True), (129, 10001, 700, 128, 64, False),
    (33, 3001, 12001, 128, 64, True), (129, 14000, 48, 128, 128, False), (65, 6000, 12001, 128, 128, True),
    (257, 14000, 48, 128, 256, False), (400, 3001, 12001, 128, 256, True), (513, 14000, 48, 192, 256, False),
    (513, 4001, 12001, 192, 256, True), (1100, 10001, 48, 224, 256, False), (257, 14000, 12001, 224, 256, True),
    (1500, 10001, 48, 256, 256, False), (1100, 4000, 14336, 256, 256, True),
]


@pytest.mark.parametrize("B,N,K,rows,tokens,split", VARIANTS)
def test_int8_gemm_every_tile(lq, B, N, K, rows, tokens, split):
    """Each tile, with and without a split reduction, on sizes that end inside tiles and steps: some
    tokens and outputs (the first and last tiles among them) against the oracle, bf16 and fp32."""
    rng = np.random.default_rng(B + N + K)
    buf = torch.randint(-128, 128, (N, pad16(K)), dtype=torch.int8, device=DEV,
                        generator=torch.Generator(DEV).manual_seed(B))
    w = buf[:, :K]
    r, bias = randn(rng, N).abs() * 1e-3, randn(rng, N)
    layer = lq.int8_layer_struct(N, K, w, r, bias=bias)
    plan = lq.lq_int8_gemm_plan(layer, B)
    assert (plan["rows"], plan["tokens"], plan["ksplit"] > 1) == (rows, tokens, split), plan
    q = make_q(rng, B, K)
    scale = randn(rng, B).abs()
    bs = np.unique(np.concatenate([np.arange(min(B, 20)), rng.integers(0, B, 30), np.arange(max(0, B - 20), B)]))
    ns = np.unique(np.concatenate([np.arange(min(N, 70)), rng.integers(0, N, 200), np.arange(max(0, N - 270), N)]))
    want = ref.product(q.cpu().numpy()[bs], host64(scale)[bs], w[torch.from_numpy(ns).to(DEV)].cpu().numpy(),
                       host64(r)[ns], host64(bias)[ns])
    for dtype in (F32, BF):
        out = torch.full((B + 2, N), 9.0, dtype=dtype, device=DEV)
        note(f"lq_int8_gemm B={B} N={N} K={K} y={dtype} {plan}")
        lq.lq_int8_gemm(layer, q, scale, B, out[1:B + 1], garbage(lq.lq_int8_gemm_workspace_size(layer, B)))
        torch.cuda.synchronize()
        assert torch.all(out[0] == 9.0) and torch.all(out[B + 1] == 9.0)
        y = out[1:B + 1]
        assert torch.isfinite(y).all()
        check_product(y[torch.from_numpy(bs).to(DEV)][:, torch.from_numpy(ns).to(DEV)], want,
                      bias[torch.from_numpy(ns).to(DEV)], dtype)


def test_int8_gemm_scales_zero_and_nan(lq):
    rng = np.random.default_rng(2)
    for B in (3, 150):
        layer, keep = make_layer(lq, rng, 70, 200)
        q = make_q(rng, B, 200)
        scale = torch.ones(B, device=DEV)
        scale[0] = 0.0
        scale[B - 1] = float("nan")
        y = torch.empty(B, 70, device=DEV)
        n = lq.lq_int8_gemm_workspace_size(layer, B)
        lq.lq_int8_gemm(layer, q, scale, B, y, garbage(n))
        torch.cuda.synchronize()
        assert torch.all(y[0] == 0) and torch.all(torch.isnan(y[B - 1])) and not torch.isnan(y[:B - 1]).any()


def test_int8_gemm_more_rows_than_b(lq):
    """Rows behind the B that are asked for stay as they were."""
    rng = np.random.default_rng(5)
    layer, keep = make_layer(lq, rng, 96, 320)
    q = make_q(rng, 300, 320)
    scale = torch.ones(300, device=DEV)
    for B in (0, 1, 17, 131):
        y = torch.full((300, 96), 5.0, device=DEV)
        lq.lq_int8_gemm(layer, q, scale, B, y, garbage(lq.lq_int8_gemm_workspace_size(layer, B)))
        torch.cuda.synchronize()
        assert torch.all(y[B:] == 5.0)
        if B:
            check_product(y[:B], ref.product(q[:B].cpu().numpy(), np.ones(B), keep[1].cpu().numpy(),
                                             host64(keep[2])), None, F32)


# ------------------------------------------------------------------ the whole layer

@pytest.mark.parametrize("xd,yd", [(F32, F32), (BF, BF), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("B,N,K", [(1, 512, 512), (2, 100, 1001), (16, 48, 8192), (40, 333, 1555), (150, 520, 700),
                                   (1, 4096, 14336), (9, 64, 17000)])
def test_int8_linear(lq, B, N, K, xd, yd):
    """The codes are exact, so the layer is as exact as the product (the scale rounds once more)."""
    rng = np.random.default_rng(N + K)
    layer, keep = make_layer(lq, rng, N, K, bias=True)
    x = randn(rng, B, K + 5).to(xd)[:, 3:3 + K]
    n = lq.lq_int8_linear_workspace_size(layer, B, xd)
    ws = garbage(n)
    y = torch.empty(B, N, dtype=yd, device=DEV)
    note(f"lq_int8_linear B={B} N={N} K={K} x={xd} y={yd}")
    lq.lq_int8_linear(layer, x, B, y, ws)
    torch.cuda.synchronize()
    assert torch.all(ws[:lq.LQ_WS_CONTROL_BYTES] == 0xA5)      # another call's control words
    q, s = ref.codes(host64(x))
    _, w, r, b, _ = keep
    check_product(y, ref.product(q, s, w.cpu().numpy(), host64(r), host64(b)), b, yd)


@pytest.mark.parametrize("B", [1, 16, 100])
def test_int8_linear_with_the_transform(lq, B):
    """Against the product of the rows that lq_quant_rows gives (checked above): the same bits."""
    rng = np.random.default_rng(B)
    N, K, hb = 272, 5120, 1024
    c = randn(rng, K).abs() + 0.5
    layer, keep = make_layer(lq, rng, N, K, hb=hb, c=c)
    x = randn(rng, B, K).to(BF)
    y, y2 = (torch.empty(B, N, device=DEV) for _ in range(2))
    lq.lq_int8_linear(layer, x, B, y, garbage(lq.lq_int8_linear_workspace_size(layer, B, BF)))
    q = torch.empty(B, K, dtype=torch.int8, device=DEV)
    s = torch.empty(B, device=DEV)
    lq.lq_quant_rows(x, B, K, q, s, hb=hb, c=c)
    lq.lq_int8_gemm(layer, q, s, B, y2, garbage(lq.lq_int8_gemm_workspace_size(layer, B)))
    torch.cuda.synchronize()
    assert torch.equal(y, y2)
    want = ref.transform(host64(x), hb=hb, c=host64(c)) @ (keep[1].double().cpu().numpy() * host64(keep[2])[:, None]).T
    # (rounding to 8 bits: half a step of top / 127 on each of K values, as independent errors)
    assert np.linalg.norm(host64(y) - want) / np.linalg.norm(want) < 0.05


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N,K,hb", [(1, 1, 1), (33, 15, 1), (31, 257, 1), (500, 1000, 1), (32, 1024, 1024),
                                    (700, 4096, 128), (90, 4097, 1), (8200, 8192, 1024), (9001, 5121, 1),
                                    (8225, 9216, 512), (8192, 16384, 1), (8193, 16385, 1), (10000, 16384, 64), (33001, 700, 1), (33000, 16, 1),
                                    (8207, 1024, 1024), (9000, 256, 8), (1025, 2047, 1), (2049, 3000, 8)])
def test_int8_linear_one_token(lq, N, K, hb, dtype):
    """One token: the bits of lq_quant_rows and lq_int8_gemm one after another, whichever path it takes."""
    rng = np.random.default_rng(N + K)
    c = randn(rng, K).abs() + 0.5 if hb > 1 else None
    layer, keep = make_layer(lq, rng, N, K, bias=True, hb=hb, c=c)
    x = randn(rng, 1, K + 1).to(dtype)[:, 1:]
    out = torch.full((3, N), 9.0, device=DEV)
    note(f"lq_int8_linear B=1 N={N} K={K} hb={hb} x={dtype}")
    lq.lq_int8_linear(layer, x, 1, out[1:2], garbage(lq.lq_int8_linear_workspace_size(layer, 1, dtype)))
    torch.cuda.synchronize()
    assert torch.all(out[0] == 9.0) and torch.all(out[2] == 9.0)
    q = torch.empty(1, pad16(K), dtype=torch.int8, device=DEV)[:, :K]
    s, y = torch.empty(1, device=DEV), torch.empty(1, N, device=DEV)
    lq.lq_quant_rows(x, 1, K, q, s, hb=hb, c=c)
    lq.lq_int8_gemm(layer, q, s, 1, y, garbage(lq.lq_int8_gemm_workspace_size(layer, 1)))
    torch.cuda.synchronize()
    assert torch.equal(out[1:2], y)


def test_int8_linear_one_token_non_finite(lq):
    rng = np.random.default_rng(9)
    layer, keep = make_layer(lq, rng, 100, 600)
    for bad in (float("nan"), float("inf")):
        x = randn(rng, 1, 600)
        x[0, 599] = bad
        y = torch.zeros(1, 100, device=DEV)
        lq.lq_int8_linear(layer, x, 1, y, garbage(lq.lq_int8_linear_workspace_size(layer, 1, F32)))
        torch.cuda.synchronize()
        assert torch.isnan(y).all()
    lq.lq_int8_linear(layer, torch.zeros(1, 600, device=DEV), 1, y,
                      garbage(lq.lq_int8_linear_workspace_size(layer, 1, F32)))
    torch.cuda.synchronize()
    assert torch.all(y == 0)


def test_int8_linear_is_the_transformed_layer(lq):
    """Weights W T^-1 after T give W x: T is orthonormal with unit scales, and its own inverse."""
    rng = np.random.default_rng(6)
    N, K, hb, B = 64, 2048, 512, 4
    W = rng.standard_normal((N, K))
    Wt = ref.transform(W, hb=hb)
    q, s = ref.codes(Wt)
    w = torch.from_numpy(q.astype(np.int8)).to(DEV)
    r = torch.from_numpy(s.astype(np.float32)).to(DEV)
    c = torch.ones(K, device=DEV)
    layer = lq.int8_layer_struct(N, K, w, r, hb=hb, c=c)
    x = randn(rng, B, K)
    x[:, 17] = 60.0                            # an outlier channel, which T spreads
    y = torch.empty(B, N, device=DEV)
    lq.lq_int8_linear(layer, x, B, y, garbage(lq.lq_int8_linear_workspace_size(layer, B, F32)))
    want = host64(x) @ W.T
    # errors uniform within half a step: weights' steps are about 3.5 / 127 of a deviation, 0.8% of a weight;
    # a row's about 6 / 127 (the outlier spread over 512 adds 60 / sqrt(512) to a deviation of 1), under 1.4%
    assert np.linalg.norm(host64(y) - want) / np.linalg.norm(want) < 0.03


# ------------------------------------------------------------------ far apart, and refused

def far_rows(B, K, dtype, far):
    """B rows of K, `far` elements apart (nothing between them is touched)."""
    return torch.empty((B - 1) * far + pad16(K), dtype=dtype, device=DEV).as_strided((B, K), (far, 1))


@pytest.mark.parametrize("B", [33, 530])
def test_rows_behind_4_gb(lq, B):
    """x, w, q and y whose last rows begin past 2^32 bytes: as the same rows lying together."""
    rng = np.random.default_rng(B)
    N, K = 540, 330
    w, rs = torch.from_numpy(rng.integers(-127, 128, (N, K), dtype=np.int8)).to(DEV), randn(rng, N).abs()
    x = randn(rng, B, K).to(BF)
    q, s = rows8(B, K)[0], torch.empty(B, device=DEV)
    wn = rows8(N, K)[0]
    wn.copy_(w)
    lq.lq_quant_rows(x, B, K, q, s)
    want = torch.empty(B, N, device=DEV)
    near = lq.int8_layer_struct(N, K, wn, rs)
    n = lq.lq_int8_linear_workspace_size(near, B, BF)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    lq.lq_int8_linear(near, x, B, want, ws)
    torch.cuda.synchronize()

    wf = far_rows(N, K, torch.int8, 1 << 23)                      # 4.5 GB
    wf.copy_(w)
    layer = lq.int8_layer_struct(N, K, wf, rs)
    far = (1 << 31) // (B - 1) // 16 * 16 + 1600                  # elements: 2^32 bytes of bf16
    xf, yf = far_rows(B, K, BF, far), far_rows(B, N, F32, far)
    xf.copy_(x)
    note(f"lq_int8_linear far apart B={B} ld={far}")
    lq.lq_int8_linear(layer, xf, B, yf, ws)
    torch.cuda.synchronize()
    assert torch.equal(yf, want)
    qf = far_rows(B, K, torch.int8, 1 << 23)                      # 4.4 GB where B is 530
    sf = torch.empty_like(s)
    note(f"lq_quant_rows far apart B={B}")
    lq.lq_quant_rows(xf, B, K, qf, sf)
    torch.cuda.synchronize()
    assert torch.equal(qf, q) and torch.equal(sf, s)
    yf.zero_()
    note(f"lq_int8_gemm far apart B={B}")
    lq.lq_int8_gemm(layer, qf, sf, B, yf, ws)
    torch.cuda.synchronize()
    assert torch.equal(yf, want)


def test_tensors_of_another_device_are_refused(lq):
    rng = np.random.default_rng(31)
    layer, keep = make_layer(lq, rng, 64, 96)
    x, y = randn(rng, 2, 96), torch.zeros(2, 64, device=DEV)
    ws = torch.empty(lq.lq_int8_linear_workspace_size(layer, 2, F32), dtype=torch.uint8)
    with pytest.raises(ValueError, match="ws must be a contiguous GPU tensor"):
        lq.lq_int8_linear(layer, x, 2, y, ws)
    with pytest.raises(ValueError, match="x must be a GPU tensor"):
        lq.lq_int8_linear(layer, x.cpu(), 2, y, ws.to(DEV))
    layer.device = 1
    with pytest.raises(ValueError, match="not the current one"):
        lq.lq_int8_linear(layer, x, 2, y, ws.to(DEV))
    with pytest.raises(ValueError, match="not the current one"):
        lq.lq_int8_gemm(layer, rows8(2, 96)[0], torch.ones(2, device=DEV), 2, y, ws.to(DEV))
    assert torch.all(y == 0)


def test_shared_rows_are_refused(lq):
    """One row seen as many (a stride of zero) is no output, and no input of quant_rows."""
    x = torch.ones(1, 64, device=DEV).expand(4, 64)
    q, s = rows8(4, 64)[0], torch.empty(4, device=DEV)
    with pytest.raises(RuntimeError):
        lq.lq_quant_rows(x, 4, 64, q, s)
    with pytest.raises(RuntimeError):
        lq.lq_norm_block(4, 64, y=x.contiguous(), a=x)


def test_transform_past_the_largest_float(lq):
    """T's sums are taken before 1 / sqrt(hb): where one passes the largest float, the row is as one that
    holds an infinity."""
    x = torch.full((2, 1024), 1e36, device=DEV)
    x[1] = 1e34
    q, s = quant(lq, x, hb=1024)
    assert np.isnan(s[0]) and np.all(q[0] == 0)
    assert q[1, 0] == 127 and np.all(q[1, 1:] == 0) and abs(s[1] * 127 / 3.2e35 - 1) < 1e-6
