"""Whether the 4-bit layer of one token takes one launch (host only)."""
import ctypes
import math
from pathlib import Path

import pytest

from bit_matmul_amd._lib import LIB, LIB_PATH, LQ_BF16, LQ_OK, LQMx4Layer

P = 0x100000


def fits(K, N, T, gate, B=1, cus=256):
    """lq::mx4_token_fits."""
    fn = ctypes.CDLL(str(LIB_PATH))._ZN2lq14mx4_token_fitsElllibb
    fn.restype, fn.argtypes = ctypes.c_bool, [ctypes.c_int64] * 3 + [ctypes.c_int, ctypes.c_bool, ctypes.c_bool]
    return fn(B, N, K, cus, T, gate)


def measured():
    for line in (Path(__file__).parent.parent / "profiles" / "mx4_token_times.txt").read_text().splitlines():
        if not line.startswith("#"):
            K, N, _, hb, gate, one, two = line.split()
            yield int(K), int(N), int(hb) > 1, gate == "1", float(one), float(two)


def test_the_rule_is_near_the_faster_way():
    """Of every size and option in the file, each with both ways measured: 0.2% above the faster way on average, 15% at
    most (256 compute units; bounds a little wider). One launch up to 8192 values whatever N, T and the gate is
    11% above it on average where it loses, 85% at most."""
    ratios, taken = [], set()
    for K, N, T, gate, one, two in measured():
        way = fits(K, N, T, gate)
        ratios.append((one if way else two) / min(one, two))
        taken.add((way, T, gate))
    assert len(ratios) > 1000 and len(taken) == 8
    assert math.exp(sum(map(math.log, ratios)) / len(ratios)) < 1.004 and max(ratios) < 1.17


def test_the_rule_depends_on_what_is_made_again():
    """More outputs, T and a gate never turn two launches into one."""
    for K in (256, 1000, 2048, 4096, 5120, 8192, 12288, 16384):
        for N in (16, 4096, 10240, 28672, 57344, 131072, 1 << 20, 1 << 26):
            for T, gate in ((False, False), (True, False), (False, True), (True, True)):
                if not fits(K, N, T, gate):
                    assert not fits(K, 2 * N, T, gate) and not fits(K, N, True, True)
                    if not (T or gate):
                        assert not fits(K, N, True, False) and not fits(K, N, False, True)
    assert fits(8192, 28672, True, False) and not fits(5120, 28672, True, False)


@pytest.mark.parametrize("K", [8, 2048, 4096, 8192, 8200, 14336, 16384])
def test_one_launch_has_fewer_than_2_32_threads(K):
    waves = 4 if K <= 4096 else 8 if K <= 8192 else 16
    for log in range(1, 29):
        for N in ((1 << log) - 1, 1 << log, (1 << log) + 1):
            assert not fits(K, N, False, False) or -(-N // 16) * 64 * waves < 1 << 32


@pytest.mark.parametrize("K,N", [(512, 131072), (5120, 10240), (5120, 28672), (2560, 57344), (8192, 1 << 24), (12288, 4096)])
def test_the_workspace_holds_two_launches(K, N):
    """Without a gate one launch, with one two: the workspace is asked for before that is known."""
    n = ctypes.c_size_t()
    layer = LQMx4Layer(N=N, K=K, ldw=16 * -(-K // 32), hb=512, w=P, w_scale=P)
    assert LIB.lq_mx4_linear_workspace_size(layer, 1, LQ_BF16, ctypes.byref(n)) == LQ_OK
    gemm = ctypes.c_size_t()
    assert LIB.lq_mx4_gemm_workspace_size(layer, 1, ctypes.byref(gemm)) == LQ_OK
    assert n.value >= gemm.value + K // 2
