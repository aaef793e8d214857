"""The heads' norms and their rotation by position against the fp64 oracle.

An output is off by: the norm's sum of squares (at most dim / 8 + 8 roundings
of 2^-24, half of it after the root), the root, two products; cos and sin (an
angle off by 2^-25 turns of 2 pi and their own rounding: 4 units of 2^-24), two
products and a sum; all relative to the pair's length. Then bf16's 2^-8.
"""
import numpy as np
import pytest
import torch

from oracle import mx4_ref as ref
from tests.gpu_util import DEV, note

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lq():
    import bit_matmul_amd
    assert torch.cuda.is_available()
    return bit_matmul_amd


def host64(t):
    return t.double().cpu().numpy()


def randn(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DEV)


def freqs(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).to(DEV)


def check(got, x, pos, freq, w, norm, one_plus, eps, interleaved):
    dim, half = x.shape[2], len(freq)
    want = ref.norm_rope(host64(x), pos, freq, None if w is None else host64(w), norm, one_plus, eps, interleaved)
    plain = ref.norm_rope(host64(x), pos, freq[:0], None if w is None else host64(w), norm, one_plus, eps)
    size = np.abs(plain)
    i = np.arange(half)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    size[:, :, first] = size[:, :, second] = np.hypot(plain[:, :, first], plain[:, :, second])
    tol = size * ((8 + (dim / 16 + 8 if norm else 0)) * U32) + 2.0 ** -149
    if got.dtype == BF:
        tol = tol + (np.abs(want) + tol) * U16
    d = np.abs(host64(got) - want)
    assert np.all(d <= tol), (d / tol).max()


def run(lq, B, Hq, Hk, dim, rot, dtype=F32, norm=True, weights=True, one_plus=False, interleaved=False, eps=1e-5,
        pos_dtype=torch.int64, far=4096, pad=5, seed=0, place=False):
    """Queries, keys and values side by side in wider rows; outputs apart, or in place."""
    rng = np.random.default_rng(seed)
    H = Hq + 2 * Hk
    rows = randn(rng, B, H * dim + pad).to(dtype)
    before = rows.clone()
    q, k = rows[:, :Hq * dim].unflatten(1, (Hq, dim)), rows[:, Hq * dim:(Hq + Hk) * dim].unflatten(1, (Hk, dim))
    pos = torch.from_numpy(rng.integers(0, far, size=B)).to(pos_dtype).to(DEV)
    freq = freqs(rot)
    w_q, w_k = (1 + 0.2 * randn(rng, dim), 0.2 * randn(rng, dim)) if weights else (None, None)
    q0, k0 = q.clone(), k.clone()
    if place:
        qo, ko = q, k
    else:
        qo = torch.full((B + 1, Hq, dim), -7.0, dtype=dtype, device=DEV)
        ko = torch.full((B + 1, Hk, dim), -7.0, dtype=dtype, device=DEV)
    note(f"lq_qk_norm_rope B={B} heads={Hq}+{Hk} dim={dim} rot={rot} {dtype} norm={norm} inter={interleaved} place={place}")
    lq.lq_qk_norm_rope(pos, freq, q=q, k=k, q_out=qo[:B], k_out=ko[:B], norm=norm, w_q=w_q, w_k=w_k,
                       one_plus=one_plus, eps=eps, interleaved=interleaved)
    torch.cuda.synchronize()
    if place:
        assert torch.equal(rows[:, (Hq + Hk) * dim:], before[:, (Hq + Hk) * dim:])
    else:
        assert torch.equal(rows, before) and torch.all(qo[B] == -7) and torch.all(ko[B] == -7)
    for got, x, w in ((qo[:B], q0, w_q), (ko[:B], k0, w_k)):
        check(got, x, pos.cpu().numpy(), freq.cpu().numpy(), w, norm, one_plus, eps, interleaved)


DIMS = [(128, 128), (64, 64), (256, 256), (512, 512), (80, 80), (96, 48), (128, 32), (100, 100), (100, 60), (18, 14),
        (2, 2), (1, 0), (7, 4), (77, 30), (511, 2), (512, 510), (33, 32), (64, 0), (250, 250)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", DIMS)
def test_heads(lq, dim, rot, interleaved, dtype):
    run(lq, 3, 5, 2, dim, rot, dtype, interleaved=interleaved, seed=dim + rot)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (64, 8), (40, 8), (7, 3), (33, 33), (300, 1)])
@pytest.mark.parametrize("B", [1, 5])
def test_counts_of_heads(lq, B, Hq, Hk, dtype):
    run(lq, B, Hq, Hk, 128, 128, dtype, seed=Hq)
    run(lq, B, Hq, Hk, 64, 64, dtype, norm=False, seed=Hq)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("how", [dict(norm=False), dict(weights=False), dict(one_plus=True), dict(place=True),
                                 dict(place=True, interleaved=True, norm=False), dict(pos_dtype=torch.int32),
                                 dict(far=1 << 31), dict(far=1 << 20, interleaved=True), dict(eps=1e-12), dict(eps=10.0)])
def test_options(lq, how, dtype):
    run(lq, 37, 8, 2, 128, 96, dtype, **how)
    run(lq, 4, 6, 3, 50, 50, dtype, **how)


def test_many_tokens(lq):
    run(lq, 1500, 9, 3, 128, 128, BF)


def test_layout_with_heads_outside(lq):
    """(heads, tokens, dim) outputs, and tokens far apart."""
    rng = np.random.default_rng(4)
    B, H, dim = 6, 5, 64
    x = randn(rng, B, H, dim)
    out = torch.full((H, B, dim + 3), -7.0, device=DEV)
    pos = torch.arange(B, device=DEV)
    freq = freqs(dim)
    lq.lq_qk_norm_rope(pos, freq, q=x, q_out=out.transpose(0, 1)[:, :, :dim], norm=False)
    torch.cuda.synchronize()
    assert torch.all(out[:, :, dim:] == -7)
    check(out.transpose(0, 1)[:, :, :dim], x, pos.cpu().numpy(), freq.cpu().numpy(), None, False, False, 1e-5, False)


def test_keys_alone_and_norm_alone(lq):
    rng = np.random.default_rng(4)
    x = randn(rng, 4, 3, 48)
    out = torch.empty_like(x)
    lq.lq_qk_norm_rope(None, None, k=x, k_out=out)
    torch.cuda.synchronize()
    check(out, x, np.zeros(4), np.zeros(0), None, True, False, 1e-5, False)


def test_extremes(lq):
    """Heads of zeros, of huge values (squares pass the largest float), of tiny ones, and of NaN or infinity, which
    spoil themselves alone; negative positions."""
    rng = np.random.default_rng(8)
    x = randn(rng, 6, 4, 64)
    x[0, 0] = 0
    x[1, 1] *= 1e30
    x[1, 2, 5] = 3e38
    x[2, 0] *= 1e-30
    pos = torch.tensor([-5, 0, 7, -100000, 1 << 24, 3], device=DEV)
    freq = freqs(64)
    out = torch.empty_like(x)
    for norm in (True, False):
        lq.lq_qk_norm_rope(pos, freq, q=x, q_out=out, norm=norm, eps=1e-6)
        torch.cuda.synchronize()
        if norm:
            check(out, x, pos.cpu().numpy(), freq.cpu().numpy(), None, True, False, 1e-6, False)
        assert torch.all(out[0, 0] == 0)
    clean = out.clone()
    x[3, 1, 9] = float("nan")
    x[4, 2, 60] = float("inf")
    lq.lq_qk_norm_rope(pos, freq, q=x, q_out=out, norm=False)
    torch.cuda.synchronize()
    bad = torch.zeros_like(x, dtype=torch.bool)
    bad[3, 1, [9, 41]] = True
    bad[4, 2, [28, 60]] = True
    assert not torch.isfinite(out[bad]).any() and torch.equal(out[~bad], clean[~bad])
