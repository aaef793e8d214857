"""Refusals of the 8-bit layer's and the norms' entry points, without a GPU:
pointer arguments are fake (never dereferenced), and every call is rejected
by the host's checks or is empty."""
import ctypes

import pytest

from bit_matmul_amd._lib import (LIB, LQ_ACT_NONE, LQ_BF16, LQ_ERR_INVALID_ARG, LQ_ERR_UNSUPPORTED,
                                 LQ_ERR_WORKSPACE, LQ_F32, LQ_INT8_MAX_K, LQ_NORM_POST,
                                 LQ_NORM_PRE, LQ_OK, LQ_ROW_MAX_K, LQ_WS_CONTROL_BYTES,
                                 LQInt8Layer, LQInt8PlanInfo, LQNormBlockArgs)

P = 0x100000            # fake, 16-byte aligned device address
INV, UNS = LQ_ERR_INVALID_ARG, LQ_ERR_UNSUPPORTED

QUANT = dict(x=P, xtype=LQ_BF16, ldx=64, gate=None, ldg=0, act=LQ_ACT_NONE, B=2, K=64, hb=1, c=None,
             q=P, ldq=64, scale=P)


def quant(**kw):
    a = {**QUANT, **kw}
    return LIB.lq_quant_rows(*(a[k] for k in QUANT), None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INV), (dict(x=P + 1), INV), (dict(xtype=LQ_F32, x=P + 2), INV),
    (dict(xtype=5), INV), (dict(ldx=63), INV), (dict(gate=P, ldg=63), INV),
    (dict(gate=P + 1, ldg=64), INV), (dict(act=5), INV), (dict(act=-1), INV), (dict(B=-1), INV),
    (dict(K=0), INV), (dict(hb=0), INV), (dict(hb=3), INV), (dict(hb=128), INV),
    (dict(K=4096, ldx=4096, ldq=4096, hb=2048), UNS), (dict(c=P + 2), INV), (dict(q=None), INV),
    (dict(q=P + 8), INV), (dict(ldq=72), INV), (dict(K=65, ldx=65), INV), (dict(scale=None), INV),
    (dict(scale=P + 2), INV), (dict(B=(1 << 20) + 1), UNS), (dict(ldq=(1 << 23) + 16), UNS),
    (dict(K=LQ_ROW_MAX_K + 1, ldx=LQ_ROW_MAX_K + 1, ldq=LQ_ROW_MAX_K + 16), UNS),
    (dict(B=0), LQ_OK), (dict(B=0, x=None, q=None, scale=None), LQ_OK),
])
def test_quant_rows_validation(kw, status):
    assert quant(**kw) == status


def layer(**kw):
    a = dict(N=32, K=64, ldw=64, hb=1, reserved=0, w=P, c=None, row_scale=P, bias=None)
    return LQInt8Layer(**{**a, **kw})


LAYERS = [
    (dict(N=-1), INV), (dict(K=0), INV), (dict(ldw=48), INV), (dict(ldw=72), INV),
    (dict(K=65), INV), (dict(hb=3), INV), (dict(hb=0), INV), (dict(reserved=1), INV),
    (dict(K=LQ_INT8_MAX_K + 1, ldw=LQ_INT8_MAX_K + 1), UNS), (dict(N=(1 << 28) + 1), UNS),
    (dict(ldw=(1 << 23) + 16), UNS), (dict(N=1 << 28, K=16), LQ_OK),
]


@pytest.mark.parametrize("kw,status", LAYERS)
def test_int8_layer_validation(kw, status):
    n = ctypes.c_size_t(77)
    if status == LQ_OK:
        assert LIB.lq_int8_gemm_workspace_size(layer(**kw), 2, ctypes.byref(n)) == status
        assert LIB.lq_int8_gemm_workspace_size(layer(**kw), 1 << 10, ctypes.byref(n)) == UNS
        return
    assert LIB.lq_int8_gemm_workspace_size(layer(**kw), 2, ctypes.byref(n)) == status
    assert LIB.lq_int8_linear_workspace_size(layer(**kw), 2, LQ_F32, ctypes.byref(n)) == status
    assert LIB.lq_int8_gemm(layer(**kw), P, 64, P, 2, P, LQ_F32, 32, None, 0, None) == status
    assert LIB.lq_int8_linear(layer(**kw), P, LQ_F32, 64, 2, P, LQ_F32, 32, P, 1 << 30, None) == status
    assert n.value == 77


def test_int8_sizes():
    n = ctypes.c_size_t(77)
    assert LIB.lq_int8_gemm_workspace_size(None, 2, ctypes.byref(n)) == INV
    assert LIB.lq_int8_gemm_workspace_size(layer(), 2, None) == INV
    assert LIB.lq_int8_gemm_workspace_size(layer(), -1, ctypes.byref(n)) == INV
    assert LIB.lq_int8_linear_workspace_size(layer(), 2, 9, ctypes.byref(n)) == INV
    assert LIB.lq_int8_gemm_workspace_size(layer(K=LQ_INT8_MAX_K, ldw=LQ_INT8_MAX_K + 1), 2,
                                           ctypes.byref(n)) == LQ_OK
    # the whole layer holds a row in registers: its K stops earlier
    assert LIB.lq_int8_linear_workspace_size(layer(K=LQ_INT8_MAX_K, ldw=LQ_INT8_MAX_K + 1), 2, LQ_F32,
                                             ctypes.byref(n)) == UNS
    assert LIB.lq_int8_linear_workspace_size(layer(), 3, LQ_BF16, ctypes.byref(n)) == LQ_OK
    assert n.value >= LQ_WS_CONTROL_BYTES + 3 * 64 + 3 * 4
    assert LIB.lq_int8_linear_workspace_size(layer(), 0, LQ_BF16, ctypes.byref(n)) == LQ_OK
    assert n.value == 0


GEMM = dict(q=P, ldq=64, scale=P, B=2, y=P, ytype=LQ_BF16, ldy=32, ws=None, wsb=0)


@pytest.mark.parametrize("kw,lkw,status", [
    (dict(q=None), {}, INV), (dict(q=P + 4), {}, INV), (dict(ldq=72), {}, INV), (dict(ldq=48), {}, INV),
    (dict(scale=None), {}, INV), (dict(scale=P + 1), {}, INV), (dict(y=None), {}, INV),
    (dict(y=P + 1), {}, INV), (dict(ytype=LQ_F32, y=P + 2), {}, INV), (dict(ytype=2), {}, INV),
    (dict(ldy=31), {}, INV), (dict(B=-1), {}, INV), ({}, dict(w=None), INV), ({}, dict(w=P + 8), INV),
    ({}, dict(row_scale=None), INV), ({}, dict(bias=P + 2), INV), (dict(B=(1 << 20) + 1), {}, UNS),
    (dict(B=0), {}, LQ_OK), (dict(y=None), dict(N=0), LQ_OK),
])
def test_int8_gemm_validation(kw, lkw, status):
    a = {**GEMM, **kw}
    assert LIB.lq_int8_gemm(layer(**lkw), *(a[k] for k in GEMM), None) == status


def test_int8_gemm_plan():
    info = LQInt8PlanInfo()
    assert LIB.lq_int8_gemm_plan(layer(), 2, None) == INV
    assert LIB.lq_int8_gemm_plan(layer(), 0, ctypes.byref(info)) == INV
    assert LIB.lq_int8_gemm_plan(layer(N=0), 2, ctypes.byref(info)) == INV
    assert LIB.lq_int8_gemm_plan(layer(reserved=2), 2, ctypes.byref(info)) == INV
    n = ctypes.c_size_t()
    for B, N, K in ((1, 32, 64), (16, 8192, 28672), (2048, 8192, 28672), (3, 1 << 28, 16), (1 << 20, 1 << 16, 16)):
        lay = layer(N=N, K=K, ldw=K)
        assert LIB.lq_int8_gemm_plan(lay, B, ctypes.byref(info)) == LQ_OK
        tiles = -(-N // info.rows) * -(-B // info.tokens)
        assert info.workgroups == tiles * info.ksplit < 1 << 24
        assert 1 <= info.ksplit <= -(-K // 128)
        assert LIB.lq_int8_gemm_workspace_size(lay, B, ctypes.byref(n)) == LQ_OK
        # every part's sums, 4 bytes each, behind the control area
        assert (n.value == 0) == (info.ksplit == 1)
        if info.ksplit > 1:
            assert n.value >= LQ_WS_CONTROL_BYTES + 4 * info.workgroups * info.rows * info.tokens


def test_int8_gemm_workspace_is_checked():
    lay = layer(N=8192, K=28672, ldw=28672)
    n = ctypes.c_size_t()
    assert LIB.lq_int8_gemm_workspace_size(lay, 64, ctypes.byref(n)) == LQ_OK and n.value > 0

    def f(ws, size):
        return LIB.lq_int8_gemm(lay, P, 28672, P, 64, P, LQ_F32, 8192, ws, size, None)
    assert f(None, 0) == LQ_ERR_WORKSPACE
    assert f(P, n.value - 1) == LQ_ERR_WORKSPACE
    assert f(P + 8, n.value) == INV


def test_int8_linear_validation():
    n = ctypes.c_size_t()
    assert LIB.lq_int8_linear_workspace_size(layer(), 2, LQ_BF16, ctypes.byref(n)) == LQ_OK

    def f(x=P, xt=LQ_BF16, ldx=64, B=2, y=P, yt=LQ_BF16, ldy=32, ws=P, wsb=n.value, lay=layer()):
        return LIB.lq_int8_linear(lay, x, xt, ldx, B, y, yt, ldy, ws, wsb, None)
    assert f(x=None) == INV and f(x=P + 1) == INV and f(xt=7) == INV and f(ldx=63) == INV
    assert f(y=None) == INV and f(ldy=1) == INV and f(yt=4) == INV
    assert f(lay=layer(c=P + 1)) == INV and f(lay=layer(w=None)) == INV
    assert f(ws=None) == LQ_ERR_WORKSPACE and f(wsb=n.value - 1) == LQ_ERR_WORKSPACE
    assert f(ws=P + 4) == INV
    assert f(B=0, x=None, y=None, ws=None, wsb=0) == LQ_OK


NORM = dict(B=2, K=64, y=P, ldy=64, ytype=LQ_BF16, h=P, ldh=64, htype=LQ_BF16, h_out=P, ldh_out=64,
            a=P, lda=64, atype=LQ_BF16, alpha=1.0, eps=1e-5, flags=LQ_NORM_POST | LQ_NORM_PRE)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INV), (dict(K=0), INV), (dict(K=LQ_ROW_MAX_K + 1), UNS), (dict(B=(1 << 20) + 1), UNS),
    (dict(y=P + 1), INV), (dict(ytype=3), INV), (dict(ldy=63), INV), (dict(h=P + 1), INV),
    (dict(htype=-1), INV), (dict(ldh=63), INV), (dict(ldh_out=63), INV), (dict(atype=2), INV),
    (dict(lda=0), INV), (dict(gate=P, ldg=1), INV), (dict(gate=P + 1), INV), (dict(act=9), INV),
    (dict(gate=P, y=None, flags=0), INV), (dict(y=None), INV), (dict(y=None, h=None, flags=0), INV),
    (dict(q=P, ldq=64), INV), (dict(scale=P), INV), (dict(q=P + 8, ldq=64, scale=P), INV),
    (dict(q=P, ldq=60, scale=P), INV), (dict(a=None, h_out=None), INV), (dict(w_pre=P + 2), INV),
    (dict(w_post=P + 1), INV), (dict(eps=0.0), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(eps=1e-40), INV), (dict(eps=-1.0), INV), (dict(alpha=float("inf")), INV),
    (dict(alpha=float("nan")), INV), (dict(flags=16), INV), (dict(reserved=1), INV),
    (dict(B=0), LQ_OK),
])
def test_norm_block_validation(kw, status):
    assert LIB.lq_norm_block(LQNormBlockArgs(**{**NORM, **kw}), None) == status


def test_norm_block_null_args():
    assert LIB.lq_norm_block(None, None) == INV


def test_python_checks_name_the_argument():
    import torch

    import bit_matmul_amd as lq
    t = torch.zeros(2, 64)
    q = torch.zeros(2, 64, dtype=torch.int8)
    with pytest.raises(ValueError, match="x must be a GPU tensor"):
        lq.lq_quant_rows(t, 2, 64, q, torch.zeros(2))
    with pytest.raises(ValueError, match="w must be an int8 tensor"):
        lq.int8_layer_struct(2, 64, t, torch.zeros(2))
    with pytest.raises(ValueError, match="y must be a GPU tensor"):
        lq.lq_norm_block(2, 64, y=t)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        lq.lq_norm_block(2, 64, y=t.half())
