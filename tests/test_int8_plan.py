"""How an 8-bit layer would run (host only)."""
import ctypes
import math
from pathlib import Path

import pytest

from bit_matmul_amd import lq_int8_linear_plan
from bit_matmul_amd._lib import (LIB, LQ_ERR_INVALID_ARG, LQ_ERR_UNSUPPORTED, LQ_OK, LQ_ROW_MAX_K, LQInt8Layer,
                                 LQInt8PlanInfo)

P = 0x100000


def layer(N, K, hb=1):
    return LQInt8Layer(N=N, K=K, ldw=-(-K // 16) * 16, hb=hb, w=P, row_scale=P)


def gemm_plan(lay, B):
    info = LQInt8PlanInfo()
    assert LIB.lq_int8_gemm_plan(lay, B, ctypes.byref(info)) == LQ_OK
    return info


@pytest.mark.parametrize("K", [16, 1024, 1040, 4096, 4112])
@pytest.mark.parametrize("hb", [1, 16])
@pytest.mark.parametrize("N", [1, 40, 8192, 8193, 32769, (1 << 27) + 5, (1 << 28) - 16, (1 << 28) - 15, 1 << 28])
def test_every_launch_fits(N, K, hb):
    """A launch has fewer than 2^32 threads, 256 to a workgroup, up to the largest layer."""
    lay = layer(N, K, hb)
    p = lq_int8_linear_plan(lay, 1)
    assert p["workgroups"] * 256 < 1 << 32
    assert p["workgroups"] >= -(-N // p["rows"])
    g = gemm_plan(lay, 1)
    assert g.workgroups * 256 < 1 << 32
    if p["tokens"] != 1:
        assert (p["rows"], p["tokens"], p["ksplit"], p["workgroups"]) == (g.rows, g.tokens, g.ksplit, g.workgroups)


@pytest.mark.parametrize("N,K,hb,rows", [
    (33, 15, 1, 16), (32, 1024, 1024, 16), (700, 4096, 128, 16), (90, 4097, 1, 0), (8192, 1024, 1, 16),
    (8193, 1024, 1024, 32), (32769, 512, 1, 32), (32768, 512, 1, 16), (28672, 2048, 1024, 16), (40000, 1025, 1, 16),
    (1 << 28, 512, 1, 32), ((1 << 28) - 16, 2048, 1, 16), (1 << 28, 2048, 1, 0),
])
def test_one_token_in_one_launch(N, K, hb, rows):
    p = lq_int8_linear_plan(layer(N, K, hb), 1)
    assert (p["rows"] if p["tokens"] == 1 else 0) == rows
    assert lq_int8_linear_plan(layer(N, K, hb), 2)["tokens"] > 1


def test_linear_plan_validation():
    info, ok = LQInt8PlanInfo(), layer(32, 64)
    assert LIB.lq_int8_linear_plan(ok, 1, None) == LQ_ERR_INVALID_ARG
    assert LIB.lq_int8_linear_plan(None, 1, ctypes.byref(info)) == LQ_ERR_INVALID_ARG
    assert LIB.lq_int8_linear_plan(ok, 0, ctypes.byref(info)) == LQ_ERR_INVALID_ARG
    assert LIB.lq_int8_linear_plan(layer(0, 64), 1, ctypes.byref(info)) == LQ_ERR_INVALID_ARG
    assert LIB.lq_int8_linear_plan(layer(32, 64, 3), 1, ctypes.byref(info)) == LQ_ERR_INVALID_ARG
    assert LIB.lq_int8_linear_plan(layer(32, LQ_ROW_MAX_K + 1), 1, ctypes.byref(info)) == LQ_ERR_UNSUPPORTED
    assert LIB.lq_int8_linear_plan(ok, 1, ctypes.byref(info)) == LQ_OK


def test_the_plan_is_near_the_best_measured():
    """Of the tiles and splits measured on one card, the plan's is 0.8% above the best on average, 12% at most
    (256 compute units; bounds a little wider)."""
    ratios = []
    for line in (Path(__file__).parent.parent / "profiles" / "int8_product_times.txt").read_text().splitlines():
        if line.startswith("#"):
            continue
        B, N, K, *times = line.split()
        times = dict(t.split("=") for t in times)
        g = gemm_plan(layer(int(N), int(K)), int(B))
        mine = times.get(f"{g.rows}x{g.tokens}/{g.ksplit}")
        if mine is not None:
            ratios.append(float(mine) / min(map(float, times.values())))
    assert len(ratios) > 170
    assert math.exp(sum(map(math.log, ratios)) / len(ratios)) < 1.012 and max(ratios) < 1.14
