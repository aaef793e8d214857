"""Refusals of the 4-bit layer's and of the heads' entry points, without a GPU:
pointer arguments are fake (never dereferenced), and every call is rejected by
the host's checks or is empty."""
import ctypes

import pytest

from bit_matmul_amd._lib import (LIB, LQ_ACT_NONE, LQ_BF16, LQ_ERR_INVALID_ARG, LQ_ERR_UNSUPPORTED,
                                 LQ_ERR_WORKSPACE, LQ_F32, LQ_MX4_MAX_K, LQ_OK, LQ_QK_INTERLEAVED,
                                 LQ_QK_MAX_DIM, LQ_QK_NORM, LQ_WS_CONTROL_BYTES, LQMx4Layer,
                                 LQMx4PlanInfo, LQQkNormRopeArgs)

P = 0x100000            # fake, 16-byte aligned device address
INV, UNS = LQ_ERR_INVALID_ARG, LQ_ERR_UNSUPPORTED

QUANT = dict(x=P, xtype=LQ_BF16, ldx=64, gate=None, ldg=0, act=LQ_ACT_NONE, B=2, K=64, hb=1, c=None,
             q=P, ldq=32, scale=P)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INV), (dict(x=P + 1), INV), (dict(xtype=LQ_F32, x=P + 2), INV),
    (dict(xtype=5), INV), (dict(ldx=63), INV), (dict(gate=P, ldg=63), INV),
    (dict(gate=P + 1, ldg=64), INV), (dict(act=5), INV), (dict(act=-1), INV), (dict(B=-1), INV),
    (dict(K=0), INV), (dict(hb=0), INV), (dict(hb=3), INV), (dict(hb=128), INV),
    (dict(K=4096, ldx=4096, ldq=2048, hb=2048), UNS), (dict(c=P + 2), INV), (dict(q=None), INV),
    (dict(q=P + 8), INV), (dict(ldq=40), INV), (dict(ldq=16), INV), (dict(K=65, ldx=65), INV), (dict(scale=None), INV),
    (dict(scale=P + 8), INV), (dict(B=(1 << 28) + 1), UNS), (dict(ldq=(1 << 23) + 16), UNS),
    (dict(K=LQ_MX4_MAX_K + 1, ldx=LQ_MX4_MAX_K + 1, ldq=LQ_MX4_MAX_K + 16), UNS),
    (dict(B=0), LQ_OK), (dict(B=0, x=None, q=None, scale=None), LQ_OK),
])
def test_quant_rows_validation(kw, status):
    a = {**QUANT, **kw}
    assert LIB.lq_mx4_quant_rows(*(a[k] for k in QUANT), None) == status


def layer(**kw):
    a = dict(N=32, K=64, ldw=32, hb=1, reserved=0, w=P, w_scale=P, c=None, row_scale=P, bias=None)
    return LQMx4Layer(**{**a, **kw})


LAYERS = [
    (dict(N=-1), INV), (dict(K=0), INV), (dict(ldw=16), INV), (dict(ldw=40), INV),
    (dict(K=65), INV), (dict(hb=3), INV), (dict(hb=0), INV), (dict(reserved=1), INV),
    (dict(K=LQ_MX4_MAX_K + 1, ldw=1 << 20), UNS), (dict(N=(1 << 28) + 1), UNS),
    (dict(ldw=(1 << 23) + 16), UNS), (dict(N=1 << 28, K=16), LQ_OK),
]


@pytest.mark.parametrize("kw,status", LAYERS)
def test_layer_validation(kw, status):
    n = ctypes.c_size_t(77)
    if status == LQ_OK:
        assert LIB.lq_mx4_gemm_workspace_size(layer(**kw), 2, ctypes.byref(n)) == status
        assert LIB.lq_mx4_gemm_workspace_size(layer(**kw), 1 << 10, ctypes.byref(n)) == UNS
        return
    info = LQMx4PlanInfo()
    assert LIB.lq_mx4_gemm_workspace_size(layer(**kw), 2, ctypes.byref(n)) == status
    assert LIB.lq_mx4_linear_workspace_size(layer(**kw), 2, LQ_F32, ctypes.byref(n)) == status
    assert LIB.lq_mx4_gemm_plan(layer(**kw), 2, ctypes.byref(info)) == status
    assert LIB.lq_mx4_gemm(layer(**kw), P, 32, P, 2, P, LQ_F32, 32, None, 0, None) == status
    assert LIB.lq_mx4_linear(layer(**kw), P, LQ_F32, 64, None, 0, 0, 2, P, LQ_F32, 32, P, 1 << 30, None) == status
    assert n.value == 77


def test_sizes():
    n = ctypes.c_size_t(77)
    for args in ((-1, 64), (3, 0)):
        assert LIB.lq_mx4_scale_size(*args, ctypes.byref(n)) == INV
    assert LIB.lq_mx4_scale_size(3, 64, None) == INV
    assert LIB.lq_mx4_scale_size((1 << 28) + 1, 64, ctypes.byref(n)) == UNS
    assert LIB.lq_mx4_scale_size(1, LQ_MX4_MAX_K + 1, ctypes.byref(n)) == UNS
    assert n.value == 77
    for rows, K, want in ((0, 5, 0), (1, 1, 128), (16, 256, 128), (17, 257, 512), (1 << 28, 1 << 20, 1 << 43)):
        assert LIB.lq_mx4_scale_size(rows, K, ctypes.byref(n)) == LQ_OK and n.value == want
    assert LIB.lq_mx4_gemm_workspace_size(None, 2, ctypes.byref(n)) == INV
    assert LIB.lq_mx4_gemm_workspace_size(layer(), 2, None) == INV
    assert LIB.lq_mx4_gemm_workspace_size(layer(), -1, ctypes.byref(n)) == INV
    assert LIB.lq_mx4_gemm_workspace_size(layer(), (1 << 20) + 1, ctypes.byref(n)) == UNS
    assert LIB.lq_mx4_linear_workspace_size(layer(), 2, 9, ctypes.byref(n)) == INV
    assert LIB.lq_mx4_linear_workspace_size(layer(), 3, LQ_BF16, ctypes.byref(n)) == LQ_OK
    assert n.value >= LQ_WS_CONTROL_BYTES + 3 * 32 + 128
    assert LIB.lq_mx4_linear_workspace_size(layer(), 0, LQ_BF16, ctypes.byref(n)) == LQ_OK and n.value == 0
    assert LIB.lq_mx4_gemm_plan(layer(), 2, None) == INV
    assert LIB.lq_mx4_gemm_plan(layer(), 0, ctypes.byref(LQMx4PlanInfo())) == INV
    assert LIB.lq_mx4_gemm_plan(layer(N=0), 1, ctypes.byref(LQMx4PlanInfo())) == INV


GEMM = dict(q=P, ldq=32, scale=P, B=2, y=P, ytype=LQ_F32, ldy=32, ws=None, ws_bytes=0)


@pytest.mark.parametrize("kw,lay,status", [
    (dict(q=None), {}, INV), (dict(q=P + 8), {}, INV), (dict(ldq=16), {}, INV), (dict(ldq=40), {}, INV),
    (dict(scale=None), {}, INV), (dict(scale=P + 4), {}, INV), (dict(y=None), {}, INV), (dict(y=P + 2), {}, INV),
    (dict(ytype=3), {}, INV), (dict(ldy=31), {}, INV), ({}, dict(w=None), INV), ({}, dict(w=P + 8), INV),
    ({}, dict(w_scale=None), INV), ({}, dict(w_scale=P + 8), INV), ({}, dict(row_scale=P + 2), INV),
    ({}, dict(bias=P + 2), INV), (dict(B=-1), {}, INV), (dict(ldq=(1 << 23) + 16), {}, UNS),
    (dict(B=0, q=None, y=None, scale=None), {}, LQ_OK), (dict(q=None, y=None), dict(N=0), LQ_OK),
])
def test_gemm_validation(kw, lay, status):
    a = {**GEMM, **kw}
    assert LIB.lq_mx4_gemm(layer(**lay), *(a[k] for k in GEMM), None) == status


LINEAR = dict(x=P, xtype=LQ_F32, ldx=64, gate=None, ldg=0, act=0, B=2, y=P, ytype=LQ_F32, ldy=32, ws=P,
              ws_bytes=1 << 30)


@pytest.mark.parametrize("kw,lay,status", [
    (dict(x=None), {}, INV), (dict(x=P + 2), {}, INV), (dict(xtype=7), {}, INV), (dict(ldx=63), {}, INV),
    (dict(gate=P, ldg=10), {}, INV), (dict(gate=P + 2, ldg=64), {}, INV), (dict(act=9), {}, INV),
    (dict(y=None), {}, INV), (dict(ldy=3), {}, INV), (dict(ws=None), {}, LQ_ERR_WORKSPACE),
    (dict(ws_bytes=100), {}, LQ_ERR_WORKSPACE), (dict(ws=P + 8), {}, INV), ({}, dict(c=P + 2), INV),
    (dict(B=0, x=None, y=None, ws=None), {}, LQ_OK),
])
def test_linear_validation(kw, lay, status):
    a = {**LINEAR, **kw}
    assert LIB.lq_mx4_linear(layer(**lay), *(a[k] for k in LINEAR), None) == status


def heads(**kw):
    a = dict(B=2, q=P, k=P, q_out=P + (1 << 16), k_out=P + (2 << 16), ldq=512, ldq_head=128, ldk=512, ldk_head=128,
             ldq_out=512, ldq_out_head=128, ldk_out=256, ldk_out_head=128, w_q=None, w_k=None, pos=P, freq=P,
             q_heads=4, k_heads=2, dim=128, rot=128, dtype=LQ_BF16, pos_bytes=8, eps=1e-5, flags=LQ_QK_NORM, reserved=0)
    return LQQkNormRopeArgs(**{**a, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV), (dict(q_out=None), INV), (dict(q_heads=0), INV), (dict(q=None, q_out=None), INV),
    (dict(k=None), INV), (dict(k_out=None), INV), (dict(q=P + 1), INV), (dict(q_out=P + 1), INV),
    (dict(dtype=LQ_F32, k=P + 2), INV), (dict(dtype=4), INV), (dict(dim=0), INV), (dict(rot=130), INV), (dict(rot=127), INV),
    (dict(rot=-2), INV), (dict(pos=None), INV), (dict(pos=P + 4), INV), (dict(pos_bytes=4, pos=P + 2), INV), (dict(pos_bytes=2), INV),
    (dict(freq=None), INV), (dict(freq=P + 4), INV), (dict(w_q=P + 1), INV), (dict(w_k=P + 2), INV),
    (dict(eps=0.0), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV),
    (dict(eps=1e-40), INV), (dict(flags=8), INV), (dict(reserved=1), INV), (dict(B=-1), INV), (dict(q_heads=-1), INV),
    (dict(ldq=-1), INV), (dict(ldq_out=511), INV), (dict(ldq_out_head=127), INV), (dict(ldq_out=0), INV),
    (dict(ldk_out=128, ldk_out_head=128), INV), (dict(q_out=P, ldq=1024, ldq_out=512), INV),
    (dict(q_out=P, ldq_head=0), INV), (dict(dim=LQ_QK_MAX_DIM + 1, ldq_out=1 << 20), UNS), (dict(B=(1 << 20) + 1), UNS),
    (dict(q_heads=(1 << 16) + 1, ldq_out=1 << 30), UNS), (dict(ldq=(1 << 40) + 1), UNS),
    (dict(B=0), LQ_OK), (dict(B=0, q=None, k=None, q_heads=0, k_heads=0, pos=None), LQ_OK),
    (dict(q=None, q_out=None, q_heads=0, k=None, k_out=None, k_heads=0), INV),
    (dict(flags=LQ_QK_INTERLEAVED | 16), INV),
])
def test_qk_norm_rope_validation(kw, status):
    assert LIB.lq_qk_norm_rope(heads(**kw), None) == status


def test_qk_norm_rope_null():
    assert LIB.lq_qk_norm_rope(None, None) == INV
