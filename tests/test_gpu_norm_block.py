"""lq_norm_block against the fp64 oracle, and the run of a block's operators.

Errors, from the arithmetic (u = 2^-24):
* a norm: each thread adds 16 C squares one after another, then 10 levels of
  additions, all positive: the sum is within (16 C + 12) u of itself and its
  root within half that; the division, root, reciprocal and the two products
  are 6 more. `norm_err(K)` is that factor.
* h' = h + alpha u: u's error, then two roundings.
* the second norm of h': its own factor, the elementwise error of h' times
  1 / rms, and that of the rms, which is at most the largest error over rms.
* bf16 outputs: eps / 2 = 2^-8 of the value more.
"""
import numpy as np
import pytest
import torch

from oracle import int8_ref as ref
from tests.gpu_util import DEV, note
from tests.test_gpu_int8 import (check_product, garbage, gate_error, host64, make_layer, near_codes,
                                 randn, rows8, untouched)

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module")
def lq():
    import bit_matmul_amd
    assert torch.cuda.is_available()
    return bit_matmul_amd


def norm_err(K):
    blocks = -(-K // 1024)
    C = 1 if blocks <= 16 else 2 if blocks <= 32 else 4
    return ((16 * C + 12) / 2 + 6) * U32


def oracle(o, y, gate, h, w_post, w_pre, alpha, eps):
    """(h', a, error of h', error of a), errors elementwise and absolute."""
    n64 = lambda t: None if t is None else host64(t)   # noqa: E731
    u, hn, a = ref.norm_block(n64(y), n64(gate), o["act"], o["first"], o["post"], n64(w_post), n64(h), alpha,
                              o["pre"], n64(w_pre), o["one_plus"], eps)
    K = hn.shape[1]
    eh = np.zeros_like(hn)
    if u is not None:
        ge = 0.0 if gate is None else gate_error(o["act"], n64(gate)) + U32
        eu = np.abs(u) * (ge + (norm_err(K) if o["post"] else 0.0))
        if o["post"] and gate is not None and o["first"]:
            eu = eu + np.abs(u) * np.max(ge)           # (the root's part: an average of squared errors)
        eh = abs(alpha) * eu + U32 * (2 * np.abs(alpha * u) + np.abs(hn)) + 1e-37
    if not o["pre"]:
        return hn, a, eh, eh
    rms = np.sqrt(np.mean(hn * hn, axis=1, keepdims=True) + eps)
    w = 1.0 if w_pre is None else np.abs(host64(w_pre) + (1.0 if o["one_plus"] else 0.0))
    ew = 0.0 if w_pre is None or not o["one_plus"] else U32
    ea = np.abs(a) * (norm_err(K) + ew + eh.max(axis=1, keepdims=True) / rms) + eh / rms * w
    return hn, a, eh, ea


def close(t, want, err):
    tol = err * 1.01 + 1e-37
    if t.dtype == BF:
        tol = tol + U16 * (np.abs(want) + tol)
    d = np.abs(host64(t) - want)
    assert np.all(d <= tol), (d.max(), np.argwhere(~(d <= tol))[:4])


def framed(B, K, dtype, ld=None):
    buf = torch.full((B + 2, ld or K), 3.0, dtype=dtype, device=DEV)
    return buf[1:B + 1, :K], buf


def frame_kept(buf, B, K):
    assert torch.all(buf[0] == 3.0) and torch.all(buf[B + 1:] == 3.0) and torch.all(buf[:, K:] == 3.0)


def run(lq, rng, B, K, yd=BF, hd=BF, ad=BF, y=True, h=True, h_out=True, a=True, q=False, gate="none", act="none",
        first=False, post=False, pre=True, one_plus=False, alpha=1.0, weights=True, ld=None, size=1.0, eps=EPS):
    o = dict(act=act, first=first, post=post, pre=pre, one_plus=one_plus)
    make = lambda dt: (randn(rng, B, (ld or K)) * size).to(dt)[:, :K]   # noqa: E731
    ty, th = make(yd) if y else None, make(hd) if h else None
    tg = None if gate == "none" else randn(rng, K).to(yd) if gate == "vector" else randn(rng, B, ld or K).to(yd)[:, :K]
    wp = randn(rng, K) if post and weights else None
    wn = randn(rng, K) if pre and weights else None
    oh, bh = framed(B, K, hd, ld)
    oa, ba = framed(B, K, ad, ld)
    oq, bq = rows8(B, K)
    scale = torch.full((B,), 7.0, device=DEV)
    note(f"lq_norm_block B={B} K={K} y={yd if y else None} h={hd if h else None} a={ad if a else None} q={q} "
         f"gate={gate} {o} alpha={alpha} ld={ld} size={size}")
    lq.lq_norm_block(B, K, y=ty, gate=tg, act=getattr(lq, "LQ_ACT_" + act.upper()), gate_first=first, post=post,
                     w_post=wp, h=th, alpha=alpha, h_out=oh if h_out else None, pre=pre, w_pre=wn, one_plus=one_plus,
                     eps=eps, a=oa if a else None, q=oq if q else None, scale=scale if q else None)
    torch.cuda.synchronize()
    alpha = float(np.float32(alpha))
    hn, an, eh, ea = oracle(o, ty, tg, th, wp, wn, alpha, float(np.float32(eps)))
    frame_kept(bh, B, K)
    frame_kept(ba, B, K)
    if h_out:
        close(oh, hn, eh)
    else:
        assert torch.all(bh == 3.0)
    if a:
        close(oa, an, ea)
    if q:
        untouched(bq, B, K)
        near_codes((oq.cpu().numpy().astype(np.int64), scale.cpu().numpy()), an, ea)


@pytest.mark.parametrize("B,K", [(1, 1), (3, 5), (2, 8), (1, 512), (2, 1023), (3, 1025), (7, 4099), (2, 8192),
                                 (2, 16385), (1, 28672), (1, 40001), (1, 65536), (257, 96)])
@pytest.mark.parametrize("yd,hd,ad", [(BF, BF, BF), (F32, F32, F32), (BF, F32, F32), (F32, BF, BF)])
def test_norm_block_sizes(lq, B, K, yd, hd, ad):
    rng = np.random.default_rng(K + B)
    run(lq, rng, B, K, yd, hd, ad, post=True, gate="rows", act="silu")


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("gate", ["vector", "rows"])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("post", [False, True])
def test_norm_block_gates(lq, act, gate, first, post):
    run(lq, np.random.default_rng(1), 3, 1201, F32, F32, F32, gate=gate, act=act, first=first, post=post, alpha=-0.22)


@pytest.mark.parametrize("kw", [
    dict(y=False), dict(h=False), dict(h=False, alpha=0.5, post=True), dict(pre=False), dict(pre=False, a=False),
    dict(a=False, q=True), dict(q=True), dict(h_out=False), dict(weights=False, post=True), dict(one_plus=True, post=True),
    dict(alpha=0.0), dict(y=False, pre=False), dict(pre=False, a=False, q=True), dict(y=False, a=False, q=True),
    dict(eps=1e-30), dict(eps=3.0, post=True), dict(ld=2777, post=True, q=True, gate="rows", act="sigmoid"),
])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_norm_block_parts(lq, kw, dtype):
    run(lq, np.random.default_rng(2), 3, 1777, dtype, dtype, dtype, **kw)


@pytest.mark.parametrize("size", [1e-18, 1e18, 1e25, 3e36])
def test_norm_block_extreme_values(lq, size):
    """Values whose squares pass the largest float, and ones whose squares vanish next to eps."""
    run(lq, np.random.default_rng(3), 2, 3000, F32, F32, F32, size=size)
    run(lq, np.random.default_rng(4), 2, 70, F32, F32, F32, size=size, y=False)
    run(lq, np.random.default_rng(5), 2, 3000, F32, F32, F32, size=size, post=True, h=False)


def test_norm_block_zero_rows(lq):
    B, K = 3, 600
    y = torch.zeros(B, K, device=DEV)
    h = torch.zeros(B, K, device=DEV)
    h[2] = 1.0
    a, q, s = torch.empty(B, K, device=DEV), torch.empty(B, 608, dtype=torch.int8, device=DEV), torch.empty(B, device=DEV)
    lq.lq_norm_block(B, K, y=y, h=h, post=True, pre=True, a=a, q=q[:, :K], scale=s)
    torch.cuda.synchronize()
    assert torch.all(a[:2] == 0) and torch.all(q[:2] == 0) and torch.all(s[:2] == 0)
    assert torch.all(q[2, :K] == 127)


def test_norm_block_non_finite_rows(lq):
    """A row that holds a NaN or an infinity spoils no other row; its codes say NaN."""
    B, K = 4, 2500
    rng = np.random.default_rng(7)
    h = randn(rng, B, K)
    ok = h.clone()
    h[1, 77], h[2, 2499] = float("nan"), float("inf")
    a, q, s = torch.empty(B, K, device=DEV), torch.zeros(B, 2512, dtype=torch.int8, device=DEV), torch.empty(B, device=DEV)
    lq.lq_norm_block(B, K, h=h, pre=True, a=a, q=q[:, :K], scale=s)
    a2 = torch.empty(B, K, device=DEV)
    lq.lq_norm_block(B, K, h=ok, pre=True, a=a2)
    torch.cuda.synchronize()
    assert torch.equal(a[0], a2[0]) and torch.equal(a[3], a2[3])
    assert torch.all(torch.isnan(a[1])) and torch.isnan(a[2, 2499])
    assert torch.isnan(s[1]) and torch.isnan(s[2]) and torch.all(q[1:3] == 0)
    assert torch.all(torch.isfinite(s[[0, 3]]))


def test_norm_block_in_place(lq):
    """h_out = h and a = y: as with outputs of their own."""
    rng = np.random.default_rng(9)
    B, K = 5, 3333
    y, h, w = randn(rng, B, K), randn(rng, B, K), randn(rng, K)
    h1, a1 = torch.empty_like(h), torch.empty_like(y)
    lq.lq_norm_block(B, K, y=y, h=h, post=True, w_post=w, h_out=h1, pre=True, w_pre=w, a=a1)
    lq.lq_norm_block(B, K, y=y, h=h, post=True, w_post=w, h_out=h, pre=True, w_pre=w, a=y)
    torch.cuda.synchronize()
    assert torch.equal(h, h1) and torch.equal(y, a1)


def test_norm_block_empty(lq):
    lq.lq_norm_block(0, 64, y=torch.empty(0, 64, device=DEV), h=torch.empty(0, 64, device=DEV),
                     a=torch.empty(0, 64, device=DEV))


# ------------------------------------------------------------------ together

class Mlp:
    """norm to 8 bits, gate and up in one product, gated rows, down, and the next block's norm."""

    def __init__(self, lq, rng, K, F, hd):
        self.lq, self.K, self.F, self.hd = lq, K, F, hd
        self.gate_up, self.k1 = make_layer(lq, rng, 2 * F, K)
        self.down, self.k2 = make_layer(lq, rng, K, F, bias=True)
        self.w1, self.w2 = randn(rng, K) * 0.1 + 1, randn(rng, K) * 0.1 + 1

    def buffers(self, B):
        e = lambda *s, dt=F32: torch.empty(*s, dtype=dt, device=DEV)   # noqa: E731
        p = lambda K: -(-K // 16) * 16                                # noqa: E731
        lq = self.lq
        n = max(lq.lq_int8_gemm_workspace_size(l, B) for l in (self.gate_up, self.down))
        return dict(q1=e(B, p(self.K), dt=torch.int8)[:, :self.K], s1=e(B), gu=e(B, 2 * self.F, dt=self.hd),
                    q2=e(B, p(self.F), dt=torch.int8)[:, :self.F], s2=e(B), y=e(B, self.K, dt=self.hd),
                    h=e(B, self.K, dt=self.hd), a=e(B, self.K, dt=self.hd), ws=garbage(n) if n else None)

    def __call__(self, x, B, b, stream=None):
        lq, K, F = self.lq, self.K, self.F
        lq.lq_norm_block(B, K, h=x, pre=True, w_pre=self.w1, q=b["q1"], scale=b["s1"], stream=stream)
        lq.lq_int8_gemm(self.gate_up, b["q1"], b["s1"], B, b["gu"], b["ws"], stream=stream)
        lq.lq_quant_rows(b["gu"][:, F:], B, F, b["q2"], b["s2"], gate=b["gu"][:, :F], act=lq.LQ_ACT_SILU, stream=stream)
        lq.lq_int8_gemm(self.down, b["q2"], b["s2"], B, b["y"], b["ws"], stream=stream)
        lq.lq_norm_block(B, K, y=b["y"], post=True, w_post=self.w2, h=x, alpha=0.5, h_out=b["h"], pre=True,
                         w_pre=self.w1, a=b["a"], stream=stream)


@pytest.mark.parametrize("hd", [F32, BF])
@pytest.mark.parametrize("B", [1, 24, 140])
def test_mlp_run(lq, B, hd):
    """Each step against the oracle on what the step before it wrote."""
    rng = np.random.default_rng(B)
    K, F = 520, 1100
    m = Mlp(lq, rng, K, F, hd)
    x = randn(rng, B, K).to(hd)
    b = m.buffers(B)
    note(f"mlp B={B} {hd}")
    m(x, B, b)
    torch.cuda.synchronize()
    off = dict(act="none", first=False, post=False, pre=True, one_plus=False)
    _, a0, _, ea = oracle(off, None, None, x, None, m.w1, 1.0, float(np.float32(1e-5)))
    near_codes((b["q1"].cpu().numpy().astype(np.int64), b["s1"].cpu().numpy()), a0, ea)
    want = ref.product(b["q1"].cpu().numpy(), host64(b["s1"]), m.k1[1].cpu().numpy(), host64(m.k1[2]))
    check_product(b["gu"], want, None, hd)
    gu = host64(b["gu"])
    v = ref.transform(gu[:, F:], gu[:, :F], "silu")
    near_codes((b["q2"].cpu().numpy().astype(np.int64), b["s2"].cpu().numpy()), v, (np.abs(v) + 1e-30) * 18 * U32)
    want = ref.product(b["q2"].cpu().numpy(), host64(b["s2"]), m.k2[1].cpu().numpy(), host64(m.k2[2]), host64(m.k2[3]))
    check_product(b["y"], want, m.k2[3], hd)
    hn, an, eh, ea = oracle({**off, "post": True}, b["y"], None, x, m.w2, m.w1, 0.5, float(np.float32(1e-5)))
    close(b["h"], hn, eh)
    close(b["a"], an, ea)


@pytest.mark.parametrize("B", [1, 20, 140])
def test_mlp_captured_and_replayed(lq, B):
    """A captured run replayed on new inputs, with eager work between the replays: the same bits."""
    rng = np.random.default_rng(B + 1)
    m = Mlp(lq, rng, 520, 1100, BF)
    x = randn(rng, B, 520).to(BF)
    b, e = m.buffers(B), m.buffers(B)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m(x, B, b)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m(x, B, b)
    for i in range(4):
        x.copy_(randn(rng, B, 520).to(BF))
        m(x, B, e)
        want = {k: e[k].clone() for k in ("h", "a", "y", "gu")}
        if i % 2:
            torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k, t in want.items():
            assert torch.equal(b[k], t), (i, k)


def test_mlp_on_two_streams(lq):
    """Two runs at once, each with its own buffers and stream, equal the runs one after another."""
    rng = np.random.default_rng(12)
    m = Mlp(lq, rng, 1040, 2200, BF)
    xs = [randn(rng, B, 1040).to(BF) for B in (150, 9)]
    want = []
    for x in xs:
        b = m.buffers(x.shape[0])
        m(x, x.shape[0], b)
        want.append(b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [m.buffers(x.shape[0]) for x in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        for x, b, st in zip(xs, got, streams):
            m(x, x.shape[0], b, stream=st)
    torch.cuda.synchronize()
    for b, w in zip(got, want):
        assert torch.equal(b["a"], w["a"]) and torch.equal(b["h"], w["h"])
