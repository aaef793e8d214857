"""Calls of the 8-bit rows, the norms and the 8-bit layer that the other files leave out: long rows with T and a
gate or into 8-bit rows, layers captured into graphs that share a workspace, and calls from two threads."""
import threading

import numpy as np
import pytest
import torch

from oracle import int8_ref as ref
from tests.gpu_util import DEV, note
from tests.test_gpu_int8 import BF, F32, U32, garbage, gate_error, host64, make_layer, near_codes, quant, randn, rows8
from tests.test_gpu_norm_block import run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lq():
    import bit_matmul_amd
    assert torch.cuda.is_available()
    return bit_matmul_amd


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("act", [None, "silu", "gelu"])
@pytest.mark.parametrize("K,hb", [(17408, 1024), (20480 + 8, 8), (33792, 1024), (65536, 512)])
def test_long_rows_with_gate_and_transform(lq, K, hb, act, dtype):
    """Two and four blocks of 1024 a wavefront. T's error as in test_gpu_int8, the gate's on each of its sums."""
    rng = np.random.default_rng(K + hb)
    B = 2
    x, c = randn(rng, B, K).to(dtype), randn(rng, K).abs() + 0.5
    g = None if act is None else randn(rng, B, K).to(dtype)
    u = ref.transform(host64(x), None if g is None else host64(g), act or "none")
    v = ref.transform(u, hb=hb, c=host64(c))
    each = 0.0 if g is None else np.max(gate_error(act, host64(g))) + U32
    tot = np.abs(u * host64(c)).reshape(B, -1, hb).sum(axis=2, keepdims=True) / np.sqrt(hb)
    err = np.broadcast_to((each + (np.log2(hb) + 2) * U32) * tot, (B, K // hb, hb)).reshape(B, K)
    near_codes(quant(lq, x, g, act or "none", hb, c), v, err)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("K", [16400, 32768, 40001])
def test_long_norms_into_8_bit_rows(lq, K, dtype):
    run(lq, np.random.default_rng(K), 2, K, dtype, dtype, dtype, q=True, post=True, gate="rows", act="silu", first=True)


@pytest.mark.parametrize("K", [20000, 40001])
def test_long_norms_in_place(lq, K):
    rng = np.random.default_rng(K)
    y, h, w = randn(rng, 3, K), randn(rng, 3, K), randn(rng, K)
    h1, a1 = torch.empty_like(h), torch.empty_like(y)
    lq.lq_norm_block(3, K, y=y, h=h, post=True, w_post=w, h_out=h1, pre=True, w_pre=w, a=a1)
    lq.lq_norm_block(3, K, y=y, h=h, post=True, w_post=w, h_out=h, pre=True, w_pre=w, a=y)
    torch.cuda.synchronize()
    assert torch.equal(h, h1) and torch.equal(y, a1)


# one launch; rows and few tokens; a split reduction and its join; tiles
LAYERS = [(1, 300, 2048, 512), (1, 200, 9216, 1024), (40, 260, 12288, 1024), (300, 520, 1536, 1)]


def test_layers_captured_with_one_workspace(lq):
    """A graph for each layer, all with one workspace, replayed in turn on new inputs with eager calls between
    them: the eager bits."""
    rng = np.random.default_rng(0)
    runs = []
    for B, N, K, hb in LAYERS:
        layer, keep = make_layer(lq, rng, N, K, bias=True, hb=hb, c=randn(rng, K).abs() + 0.5 if hb > 1 else None)
        runs.append((layer, keep, randn(rng, B, K).to(BF), torch.empty(B, N, dtype=BF, device=DEV), torch.empty(B, N, dtype=BF, device=DEV)))
    sizes = [lq.lq_int8_linear_workspace_size(r[0], r[2].shape[0], BF) for r in runs]
    assert any(lq.lq_int8_linear_plan(r[0], r[2].shape[0])["ksplit"] > 1 for r in runs)
    ws, ws2 = garbage(max(sizes)), garbage(max(sizes))
    graphs = []
    for layer, _, x, y, _ in runs:
        lq.lq_int8_linear(layer, x, x.shape[0], y, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lq.lq_int8_linear(layer, x, x.shape[0], y, ws)
        graphs.append(g)
    for turn in range(3):
        for layer, _, x, y, y2 in runs:
            x.copy_(randn(rng, *x.shape).to(BF))
            y.zero_()
            lq.lq_int8_linear(layer, x, x.shape[0], y2, ws2)
        for g in graphs:
            g.replay()
        if turn:
            lq.lq_int8_linear(runs[1][0], runs[1][2], 1, runs[1][4], ws)
        torch.cuda.synchronize()
        for r in runs:
            assert torch.equal(r[3], r[4])


def test_calls_from_two_threads(lq):
    """Two threads, each with its own stream, workspace and outputs: the bits of one after another."""
    rng = np.random.default_rng(3)
    jobs = []
    for B, N, K, hb in (LAYERS[2], LAYERS[3]):
        layer, keep = make_layer(lq, rng, N, K, hb=hb, c=randn(rng, K).abs() + 0.5 if hb > 1 else None)
        x, w = randn(rng, B, K), randn(rng, K)
        n = lq.lq_int8_linear_workspace_size(layer, B, F32)
        want, a = torch.empty(B, N, device=DEV), torch.empty(B, K, device=DEV)
        lq.lq_norm_block(B, K, h=x, pre=True, w_pre=w, a=a)
        lq.lq_int8_linear(layer, a, B, want, garbage(n))
        jobs.append((layer, keep, x, w, want, torch.zeros_like(want), torch.empty_like(a), garbage(n), torch.cuda.Stream()))
    torch.cuda.synchronize()
    errors = []

    def work(layer, keep, x, w, want, y, a, ws, stream):
        try:
            for _ in range(20):
                lq.lq_norm_block(x.shape[0], x.shape[1], h=x, pre=True, w_pre=w, a=a, stream=stream)
                lq.lq_int8_linear(layer, a, x.shape[0], y, ws, stream=stream)
        except Exception as e:      # noqa: BLE001
            errors.append(e)
    note("lq_norm_block and lq_int8_linear from two threads")
    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for j in jobs:
        assert torch.equal(j[5], j[4])


@pytest.mark.parametrize("B", [1, 3])
def test_rows_behind_the_last_one_stay(lq, B):
    """Tensors of more rows than B: what lies behind them keeps its bytes."""
    rng = np.random.default_rng(B)
    K, N = 700, 90
    layer, keep = make_layer(lq, rng, N, K)
    x = randn(rng, 6, K)
    q, _ = rows8(6, K)
    s, y, a = torch.full((6,), 4.0, device=DEV), torch.full((6, N), 4.0, device=DEV), torch.full((6, K), 4.0, device=DEV)
    lq.lq_norm_block(B, K, h=x, pre=True, a=a, q=q, scale=s)
    assert torch.all(a[B:] == 4.0) and torch.all(q[B:] == 0x55) and torch.all(s[B:] == 4.0)
    q.fill_(0x55)
    s.fill_(4.0)
    lq.lq_quant_rows(x, B, K, q, s)
    assert torch.all(q[B:] == 0x55) and torch.all(s[B:] == 4.0)
    lq.lq_int8_linear(layer, x, B, y, garbage(lq.lq_int8_linear_workspace_size(layer, B, F32)))
    assert torch.all(y[B:] == 4.0) and torch.all(y[:B] != 4.0)
