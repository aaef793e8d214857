"""The 4-bit layer and the heads' norms as they are used: weights made by the library, a run of a block's
first half captured and replayed, one workspace for several graphs, threads and streams, rows far apart and
behind the last one, tensors that are refused."""
import threading

import numpy as np
import pytest
import torch

from oracle import mx4_ref as ref
from tests.gpu_util import DEV, note
from tests.test_gpu_mx4 import (BF, F32, U16, U32, Layer, Rows, host64, near_product, quant, randn, run_gemm, same,
                                width, workspace)
from tests.test_mx4_plan import inner_plan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lq():
    import bit_matmul_amd
    assert torch.cuda.is_available()
    return bit_matmul_amd


def made_layer(lq, rng, N, K, **kw):
    """A layer whose weights the library quantised, its decoded weights, and its tensors."""
    w = randn(rng, N, K) / np.sqrt(K)
    q = torch.empty(N, width(K), dtype=torch.uint8, device=DEV)
    s = torch.empty(lq.lq_mx4_scale_size(N, K), dtype=torch.uint8, device=DEV)
    lq.lq_mx4_quant_rows(w, N, K, q, s)
    code, scale = ref.quantise(host64(w))
    return lq.mx4_layer_struct(N, K, q, s, **kw), ref.decode(code, scale, K), (q, s, kw)


@pytest.mark.parametrize("B", [1, 5, 70])
def test_weights_made_by_the_library(lq, B):
    rng = np.random.default_rng(B)
    N, K = 333, 1100
    layer, w64, keep = made_layer(lq, rng, N, K)
    x = randn(rng, B, K)
    y = torch.empty(B, N, device=DEV)
    note(f"lq_mx4_linear of library-made weights B={B}")
    lq.lq_mx4_linear(layer, x, B, y, workspace(lq.lq_mx4_linear_workspace_size(layer, B, F32)))
    torch.cuda.synchronize()
    x64 = ref.decode(*ref.quantise(host64(x)), K)
    want, size = ref.product(x64, w64)
    assert np.all(np.abs(host64(y) - want) <= size * ((K / 32 + 8) * 2.0 ** -23))


class Attention:
    """norm, 4-bit QKV layer with T, heads' norms and rotation in place."""

    def __init__(self, lq, rng, B, Hq, Hk, dim, K, hb):
        self.lq, self.B, self.K, self.Hq, self.Hk, self.dim = lq, B, K, Hq, Hk, dim
        N = (Hq + 2 * Hk) * dim
        c = (0.8 + 0.4 * torch.rand(K, generator=torch.Generator().manual_seed(1))).to(DEV)
        self.layer, self.w64, self.keep = made_layer(lq, rng, N, K, hb=hb, c=c)
        self.h, self.pos = randn(rng, B, K).to(BF), torch.randint(0, 4096, (B,), device=DEV)
        self.w_pre = 1 + 0.1 * randn(rng, K)
        self.a = torch.empty(B, K, dtype=BF, device=DEV)
        self.y = torch.empty(B, N, dtype=BF, device=DEV)
        self.ws = workspace(lq.lq_mx4_linear_workspace_size(self.layer, B, BF))
        self.freq = (10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)).to(DEV)
        self.w_q, self.w_k = 1 + 0.1 * randn(rng, dim), 1 + 0.1 * randn(rng, dim)
        self.q = self.y[:, :Hq * dim].unflatten(1, (Hq, dim))
        self.k = self.y[:, Hq * dim:(Hq + Hk) * dim].unflatten(1, (Hk, dim))

    def project(self):
        self.lq.lq_norm_block(self.B, self.K, h=self.h, pre=True, w_pre=self.w_pre, a=self.a)
        self.lq.lq_mx4_linear(self.layer, self.a, self.B, self.y, self.ws)

    def turn(self):
        self.lq.lq_qk_norm_rope(self.pos, self.freq, q=self.q, k=self.k, q_out=self.q, k_out=self.k, w_q=self.w_q,
                                w_k=self.w_k)

    def run(self):
        self.project()
        self.turn()


@pytest.mark.parametrize("B", [1, 9, 200])
def test_a_run_captured_and_replayed(lq, B):
    """The steps against the oracle, each on the one's outputs before it, then the whole as a graph with eager work
    between the replays: the eager bits."""
    rng = np.random.default_rng(B)
    at = Attention(lq, rng, B, 6, 2, 64, 1024, 512)
    note(f"norm, 4-bit layer, heads B={B}")
    at.project()
    torch.cuda.synchronize()
    code, scale = quant(lq, at.a, hb=512, c=at.keep[2]["c"])
    want, size = ref.product(ref.decode(code, scale, 1024), at.w64)
    tol = size * ((1024 / 32 + 8) * 2.0 ** -23)
    assert np.all(np.abs(host64(at.y) - want) <= tol + (np.abs(want) + tol) * U16)
    before = at.y.clone()
    at.turn()
    torch.cuda.synchronize()
    heads = host64(before).reshape(B, -1, 64)
    turned = np.concatenate([ref.norm_rope(heads[:, :6], at.pos.cpu().numpy(), at.freq.cpu().numpy(), host64(at.w_q)),
                             ref.norm_rope(heads[:, 6:8], at.pos.cpu().numpy(), at.freq.cpu().numpy(), host64(at.w_k))], axis=1)
    got = host64(at.y).reshape(B, -1, 64)
    big = np.hypot(turned[:, :, :32], turned[:, :, 32:])
    tol = np.concatenate([big, big], axis=2) * 20 * U32
    assert np.all(np.abs(got[:, :8] - turned) <= tol + (np.abs(turned) + tol) * U16)
    assert np.array_equal(got[:, 8:], heads[:, 8:])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        at.run()
    for _ in range(3):
        at.h.copy_(randn(rng, B, 1024).to(BF))
        at.pos.copy_(torch.randint(0, 1 << 20, (B,), device=DEV))
        at.run()
        eager = at.y.clone()
        at.y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(at.y, eager)


# (kernel of the plan's table, split or not, tokens, outputs, inputs)
KERNELS = [(0, False, 517, 19805, 220), (0, True, 223, 19076, 14487), (1, False, 690, 16432, 201), (1, True, 193, 17819, 14442),
           (2, False, 521, 13475, 262), (2, True, 216, 18424, 14253), (3, False, 65, 18401, 1602), (3, True, 65, 8724, 13641),
           (4, False, 68, 16664, 201), (5, False, 2, 23126, 9002), (5, True, 33, 4161, 15204), (6, False, 34, 10332, 203),
           (6, True, 35, 1448, 12967), (7, False, 1, 12372, 790), (7, True, 33, 686, 8790), (8, False, 18, 41, 211),
           (9, False, 17, 41, 263), (9, True, 17, 40, 6851), (10, False, 3, 140, 2200), (11, False, 5, 141, 2227),
           (12, False, 9, 145, 2210), (13, False, 9, 5274, 205)]


@pytest.mark.parametrize("tile,split,B,N,K", KERNELS)
def test_every_kernel_of_the_plan(lq, tile, split, B, N, K):
    """Sampled tokens and outputs (the first and last ones among them) against the oracle, fp32 and bf16, with
    garbage past K and in the scales of rows and blocks that are none."""
    plan = inner_plan(B, N, K)
    assert (plan.tile, plan.ksplit > 1) == (tile, split), (plan.tile, plan.ksplit)
    g = torch.Generator(DEV).manual_seed(N)
    units, nb = -(-K // 256), -(-K // 32)

    def side(rows):
        codes = torch.randint(0, 256, (rows, width(K) + 16), dtype=torch.uint8, device=DEV, generator=g)
        scale = torch.randint(124, 131, (-(-rows // 16) * units * 128,), dtype=torch.uint8, device=DEV, generator=g)
        places = torch.from_numpy(ref.scale_places(rows, K)[:, :nb]).to(DEV)
        none = torch.ones_like(scale, dtype=torch.bool)
        none[places.flatten()] = False
        scale[none] = 255
        return codes, scale, places

    def decoded(codes, scale, places, pick):
        return ref.decode(ref.unpack(codes[pick, :width(K)].cpu().numpy()), scale[places[pick]].cpu().numpy(), K)

    w, q = side(N), side(B)
    r, bias = torch.rand(N, device=DEV, generator=g) + 0.5, torch.randn(N, device=DEV, generator=g)
    layer = lq.mx4_layer_struct(N, K, w[0], w[1], r, bias=bias)
    rng = np.random.default_rng(B)
    bs = np.unique(np.concatenate([np.arange(min(B, 20)), rng.integers(0, B, 20), np.arange(max(0, B - 20), B)]))
    ns = np.unique(np.concatenate([np.arange(min(N, 70)), rng.integers(0, N, 150), np.arange(max(0, N - 270), N)]))
    bt, nt = torch.from_numpy(bs).to(DEV), torch.from_numpy(ns).to(DEV)
    want, size = ref.product(decoded(*q, bt), decoded(*w, nt), host64(r)[ns], host64(bias)[ns])
    tol = size * ((K / 32 + 8) * 2.0 ** -23) + 3 * U32 * (np.abs(want) + np.abs(host64(bias)[ns]))
    for dtype in (F32, BF):
        out = torch.full((B + 2, N), 9.0, dtype=dtype, device=DEV)
        note(f"lq_mx4_gemm kernel {tile} parts {plan.ksplit} B={B} N={N} K={K} y={dtype}")
        lq.lq_mx4_gemm(layer, q[0], q[1], B, out[1:B + 1], workspace(lq.lq_mx4_gemm_workspace_size(layer, B)))
        torch.cuda.synchronize()
        assert torch.all(out[0] == 9.0) and torch.all(out[B + 1] == 9.0)
        assert torch.isfinite(out).all()
        got = host64(out[1:B + 1][bt][:, nt])
        assert np.all(np.abs(got - want) <= tol + (0 if dtype == F32 else (np.abs(want) + tol) * U16))


# one launch; rows and few tokens; a split reduction and its join; tiles
LAYERS = [(1, 300, 2048, 512), (4, 200, 9216, 1024), (40, 260, 12288, 1024), (300, 520, 1536, 1)]


def small(lq, rng, B, N, K, hb):
    c = (0.8 + 0.4 * torch.rand(K, generator=torch.Generator().manual_seed(3))).to(DEV) if hb > 1 else None
    lay = Layer(lq, N, K, seed=N, bias=True, hb=hb, c=c)
    lay.c = c
    return lay


def test_layers_captured_with_one_workspace(lq):
    """A graph for each layer, all with one workspace, replayed in turn on new inputs with eager calls between
    them: the eager bits."""
    rng = np.random.default_rng(0)
    runs = [(small(lq, rng, *L), randn(rng, L[0], L[2]).to(BF), torch.empty(L[0], L[1], dtype=BF, device=DEV),
             torch.empty(L[0], L[1], dtype=BF, device=DEV)) for L in LAYERS]
    assert any(lq.lq_mx4_gemm_plan(r[0].struct, len(r[1]))["ksplit"] > 1 for r in runs)
    n = max(lq.lq_mx4_linear_workspace_size(r[0].struct, len(r[1]), BF) for r in runs)
    ws, ws2 = workspace(n), workspace(n)
    graphs = []
    for lay, x, y, _ in runs:
        lq.lq_mx4_linear(lay.struct, x, len(x), y, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lq.lq_mx4_linear(lay.struct, x, len(x), y, ws)
        graphs.append(g)
    for turn in range(3):
        for lay, x, y, y2 in runs:
            x.copy_(randn(rng, *x.shape).to(BF))
            y.zero_()
            lq.lq_mx4_linear(lay.struct, x, len(x), y2, ws2)
        for g in graphs:
            g.replay()
        if turn:
            lq.lq_mx4_linear(runs[1][0].struct, runs[1][1], len(runs[1][1]), runs[1][3], ws)
        torch.cuda.synchronize()
        for r in runs:
            assert torch.equal(r[2], r[3])


def test_calls_from_two_threads(lq):
    """Two threads, each with its own stream, workspace and outputs: the bits of one after another."""
    rng = np.random.default_rng(3)
    jobs = []
    for L in (LAYERS[2], LAYERS[3]):
        B, N, K, _ = L
        lay, x = small(lq, rng, *L), randn(rng, B, K)
        n = lq.lq_mx4_linear_workspace_size(lay.struct, B, F32)
        want = torch.empty(B, N, device=DEV)
        lq.lq_mx4_linear(lay.struct, x, B, want, workspace(n))
        heads = want[:, :N // 20 * 20].unflatten(1, (-1, 20))
        turned, freq = torch.empty_like(heads, memory_format=torch.contiguous_format), torch.rand(10, dtype=torch.float64, device=DEV)
        pos = torch.arange(B, device=DEV)
        lq.lq_qk_norm_rope(pos, freq, q=heads, q_out=turned)
        jobs.append((lay, x, pos, freq, want, turned, torch.zeros_like(want), torch.zeros_like(turned), workspace(n),
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    errors = []

    def work(lay, x, pos, freq, want, turned, y, t, ws, stream):
        try:
            for _ in range(20):
                lq.lq_mx4_linear(lay.struct, x, len(x), y, ws, stream=stream)
                lq.lq_qk_norm_rope(pos, freq, q=y[:, :lay.N // 20 * 20].unflatten(1, (-1, 20)), q_out=t, stream=stream)
        except Exception as e:      # noqa: BLE001
            errors.append(e)
    note("lq_mx4_linear and lq_qk_norm_rope from two threads")
    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for j in jobs:
        assert torch.equal(j[6], j[4]) and torch.equal(j[7], j[5])


@pytest.mark.parametrize("B", [1, 3])
def test_rows_behind_the_last_one_stay(lq, B):
    rng = np.random.default_rng(B)
    lay = Layer(lq, 90, 700)
    x, y = randn(rng, 6, 700), torch.full((6, 90), 4.0, device=DEV)
    q = torch.full((6, width(700)), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((lq.lq_mx4_scale_size(6, 700),), 0x55, dtype=torch.uint8, device=DEV)
    lq.lq_mx4_quant_rows(x, B, 700, q, s)
    lq.lq_mx4_linear(lay.struct, x, B, y, workspace(lq.lq_mx4_linear_workspace_size(lay.struct, B, F32)))
    torch.cuda.synchronize()
    own = np.zeros(len(s), dtype=bool)
    own[ref.scale_places(B, 700)] = True
    assert torch.all(q[B:] == 0x55) and np.all(s.cpu().numpy()[~own] == 0x55)
    assert torch.all(y[B:] == 4.0) and torch.all(y[:B] != 4.0)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N,K,hb", [(1, 8, 1), (33, 40, 8), (300, 2040, 1), (90, 2048, 1024), (16, 3000, 1), (300, 4096, 512),
                                    (77, 8192, 1024), (4100, 8000, 64), (130, 8200, 1), (2000, 14336, 1024), (4096, 16384, 128)])
def test_one_token_in_one_launch(lq, N, K, hb, dtype):
    """Every length of row that one launch takes, with a gate, T, a row scale and a bias and without: no rows in the
    workspace, and the product of lq_mx4_quant_rows' rows."""
    rng = np.random.default_rng(N + K)
    c = (0.8 + 0.4 * torch.rand(K, generator=torch.Generator().manual_seed(3))).to(DEV) if hb > 1 else None
    for act in (None, "gelu"):
        lay = Layer(lq, N, K, bias=act is None, row_scale=act is not None, hb=hb, c=c)
        x, g = randn(rng, 1, K).to(dtype), randn(rng, 1, K).to(dtype)
        y = torch.full((2, N), 4.0, dtype=dtype, device=DEV)
        ws = workspace(lq.lq_mx4_linear_workspace_size(lay.struct, 1, dtype))
        how = dict(gate=g, act=lq.LQ_ACT_GELU) if act else {}
        note(f"lq_mx4_linear one token N={N} K={K} hb={hb} {dtype} act={act}")
        lq.lq_mx4_linear(lay.struct, x, 1, y, ws, **how)
        torch.cuda.synchronize()
        assert torch.all(ws == 0xA5) and torch.all(y[1] == 4.0)
        code, scale = quant(lq, x, gate=g if act else None, act=act or "none", hb=hb, c=c)
        near_product(y[:1], ref.decode(code, scale, K), lay)


@pytest.mark.parametrize("N,K", [(40, 4099), (4112, 8200), (40, 20000)])
def test_one_token_in_two_launches(lq, N, K):
    """Rows not 8 values at a time, too long, or with more outputs than compute units take."""
    rng = np.random.default_rng(K)
    lay, x = Layer(lq, N, K), randn(rng, 1, K)
    y, ws = torch.empty(1, N, device=DEV), workspace(lq.lq_mx4_linear_workspace_size(lay.struct, 1, F32))
    lq.lq_mx4_linear(lay.struct, x, 1, y, ws)
    torch.cuda.synchronize()
    assert not torch.all(ws == 0xA5)
    near_product(y, ref.decode(*quant(lq, x), K), lay)


def test_one_token_holding_an_infinity(lq):
    lay, x = Layer(lq, 100, 4096), torch.ones(1, 4096, device=DEV)
    y = torch.zeros(1, 100, device=DEV)
    x[0, 77] = float("inf")
    lq.lq_mx4_linear(lay.struct, x, 1, y, workspace(lq.lq_mx4_linear_workspace_size(lay.struct, 1, F32)))
    torch.cuda.synchronize()
    assert torch.isnan(y).all()


def far_rows(rows, cols, dtype, ld):
    return torch.empty(rows * ld, dtype=dtype, device=DEV).view(rows, ld)[:, :cols]


@pytest.mark.parametrize("B", [2, 12, 530])
def test_rows_far_apart(lq, B):
    """Rows whose last ones lie past 4 GB: the bits of dense ones."""
    rng = np.random.default_rng(B)
    N, K = 540, 288
    lay, rows = Layer(lq, N, K, bias=True), Rows(B, K)
    want = run_gemm(lq, lay, rows, B, F32)
    near_product(want, rows.q64, lay)
    wf = far_rows(N, width(K), torch.uint8, 1 << 23)                     # 4.5 GB
    wf.copy_(lay.w)
    qf = far_rows(B, width(K), torch.uint8, 1 << 23)
    qf.copy_(rows.q)
    layer = lq.mx4_layer_struct(N, K, wf, lay.scale, lay.r, bias=lay.bias)
    far = (1 << 30) // (B - 1) // 16 * 16 + 1600                         # 2^32 bytes of fp32
    yf = far_rows(B, N, F32, far)
    note(f"lq_mx4_gemm far apart B={B}")
    lq.lq_mx4_gemm(layer, qf, rows.scale, B, yf, workspace(lq.lq_mx4_gemm_workspace_size(layer, B)))
    torch.cuda.synchronize()
    assert torch.equal(yf, want)
    del wf, yf
    x = randn(rng, B, K)
    xf = far_rows(B, K, F32, far)
    xf.copy_(x)
    s = torch.full((lq.lq_mx4_scale_size(B, K),), 0x55, dtype=torch.uint8, device=DEV)
    note(f"lq_mx4_quant_rows far apart B={B}")
    lq.lq_mx4_quant_rows(xf, B, K, qf, s)
    torch.cuda.synchronize()
    same((ref.unpack(qf.cpu().numpy()), s.cpu().numpy()[ref.scale_places(B, K)[:, :K // 32]]), host64(x))


def test_heads_far_apart(lq):
    """Tokens and heads whose last ones lie past 4 GB."""
    rng = np.random.default_rng(1)
    x = randn(rng, 3, 4, 32)
    pos, freq = torch.arange(3, device=DEV), torch.rand(16, dtype=torch.float64, device=DEV)
    want = torch.empty_like(x)
    lq.lq_qk_norm_rope(pos, freq, q=x, q_out=want)
    big = torch.empty((1 << 30) + 4096, dtype=F32, device=DEV)
    for strides in ((1 << 29, 64, 1), (64, (1 << 30) // 3 // 4 * 4, 1)):
        far = big.as_strided((3, 4, 32), strides)
        far.copy_(x)
        note(f"lq_qk_norm_rope far apart {strides}")
        lq.lq_qk_norm_rope(pos, freq, q=far, q_out=far)
        torch.cuda.synchronize()
        assert torch.equal(far, want)


def test_the_same_position_twice_and_shared_inputs(lq):
    """Tokens of one position, keys that are the queries' own rows, one head seen by every token (a stride of zero)
    as an input; as an output it is refused."""
    rng = np.random.default_rng(2)
    x = randn(rng, 1, 1, 64).expand(5, 3, 64)
    pos, freq = torch.full((5,), 7, device=DEV), torch.rand(32, dtype=torch.float64, device=DEV)
    q, k = torch.empty(5, 3, 64, device=DEV), torch.empty(5, 3, 64, device=DEV)
    lq.lq_qk_norm_rope(pos, freq, q=x, k=x, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert torch.equal(q, k) and torch.equal(q, q[:1, :1].expand(5, 3, 64))
    with pytest.raises(lq.LQError):
        lq.lq_qk_norm_rope(pos, freq, q=q, q_out=torch.empty(1, 1, 64, device=DEV).expand(5, 3, 64))
    with pytest.raises(lq.LQError):        # in place, but turned round
        lq.lq_qk_norm_rope(pos[:3], freq, q=q[:3], q_out=q[:3].transpose(0, 1))


def test_refusals(lq):
    rng = np.random.default_rng(31)
    lay = Layer(lq, 64, 96)
    x, y = randn(rng, 2, 96), torch.zeros(2, 64, device=DEV)
    ws = torch.empty(lq.lq_mx4_linear_workspace_size(lay.struct, 2, F32), dtype=torch.uint8)
    with pytest.raises(ValueError, match="ws must be a contiguous GPU tensor"):
        lq.lq_mx4_linear(lay.struct, x, 2, y, ws)
    with pytest.raises(ValueError, match="x must be a GPU tensor"):
        lq.lq_mx4_linear(lay.struct, x.cpu(), 2, y, ws.to(DEV))
    with pytest.raises(ValueError, match="gate must have x's dtype"):
        lq.lq_mx4_linear(lay.struct, x, 2, y, ws.to(DEV), gate=x.to(BF))
    with pytest.raises(ValueError, match="scale must be a uint8 tensor of 128 bytes"):
        lq.lq_mx4_gemm(lay.struct, Rows(2, 96).q, torch.zeros(64, dtype=torch.uint8, device=DEV), 2, y)
    with pytest.raises(ValueError, match="q must be a uint8 tensor"):
        lq.lq_mx4_gemm(lay.struct, torch.zeros(2, 48, dtype=torch.int8, device=DEV), lay.scale, 2, y)
    with pytest.raises(ValueError, match="q has shape"):
        lq.lq_mx4_quant_rows(x, 2, 96, torch.zeros(2, 32, dtype=torch.uint8, device=DEV), lay.scale)
    lay.struct.device = 1
    with pytest.raises(ValueError, match="not the current one"):
        lq.lq_mx4_linear(lay.struct, x, 2, y, ws.to(DEV))
    with pytest.raises(ValueError, match="not the current one"):
        lq.lq_mx4_gemm(lay.struct, Rows(2, 96).q, lay.scale, 2, y, ws.to(DEV))
    assert torch.all(y == 0)
    h, pos, freq = randn(rng, 3, 2, 32), torch.arange(3, device=DEV), torch.rand(16, dtype=torch.float64, device=DEV)
    out = torch.zeros_like(h)
    for match, kw in (("q or k is needed", dict()), ("q_out must be a GPU tensor", dict(q=h)),
                      ("q_out without q", dict(k=h, k_out=out, q_out=out)), ("k_out has shape", dict(k=h, k_out=out[:, :1])),
                      ("k has shape", dict(q=h, q_out=out, k=h[:2], k_out=out[:2])),
                      ("k must be torch.float32", dict(q=h, q_out=out, k=h.to(BF), k_out=out)),
                      ("q_out must be torch.float32", dict(q=h, q_out=out.to(BF))),
                      ("q or k is needed", dict(q=h.cpu(), q_out=out)), ("q_out must be a GPU tensor", dict(q=h, q_out=out.cpu())),
                      ("heads must be dense", dict(q=h[:, :, ::2], q_out=out[:, :, :16], w_q=None))):
        with pytest.raises(ValueError, match=match):
            lq.lq_qk_norm_rope(pos, freq, **kw)
    for p, f in ((pos.float(), freq), (pos, freq.float()), (pos[:2], freq), (pos.cpu(), freq), (pos, freq.cpu())):
        with pytest.raises(ValueError):
            lq.lq_qk_norm_rope(p, f, q=h, q_out=out)
    assert torch.all(out == 0)


def test_empty_calls(lq):
    lay = Layer(lq, 64, 96)
    none = torch.empty(0, 96, device=DEV)
    y = torch.full((2, 64), 3.0, device=DEV)
    lq.lq_mx4_linear(lay.struct, none, 0, y)
    lq.lq_mx4_gemm(lay.struct, torch.empty(0, 48, dtype=torch.uint8, device=DEV),
                   torch.empty(0, dtype=torch.uint8, device=DEV), 0, y)
    lq.lq_qk_norm_rope(torch.empty(0, dtype=torch.int64, device=DEV), torch.rand(16, dtype=torch.float64, device=DEV),
                       q=torch.empty(0, 2, 32, device=DEV), q_out=torch.empty(0, 2, 32, device=DEV))
    torch.cuda.synchronize()
    assert torch.all(y == 3.0)


def test_transform_near_the_largest_float(lq):
    """Sums whose values times 1 / sqrt(hb) stay among the floats are right, where the sums of the values themselves
    pass the largest; past it the block is as one that holds an infinity, and the next 1024 values know nothing of it."""
    x = torch.zeros(1, 2048, device=DEV)
    for top in (1e36, 1e34):
        x[0, :1024] = top
        code, scale = quant(lq, x, hb=1024)
        assert ref.decode(code, scale, 2048)[0, 0] == ref.decode(*ref.quantise(np.array([[32 * top]])), 1)[0, 0]
        assert np.all(code[0, 1:] == 0) and np.all(scale[0, 1:] == 0)
    x[0, :1024] = 3e38
    x[0, 1024:] = 1.0
    code, scale = quant(lq, x, hb=1024)
    assert scale[0, 0] == 255 and np.all(code[0, :32] == 0)
    assert ref.decode(code, scale, 2048)[0, 1024] == 32.0 and np.all(scale[0, 33:] == 0)
