"""The 4-bit and the heads' oracle against brute force and closed forms."""
import numpy as np
import pytest

from oracle import mx4_ref as ref


def nearest(v, e):
    """The code of one value by trial of all eight, ties to the even one."""
    a = abs(float(v)) * 2.0 ** -e
    off = [abs(a - g) for g in (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)]
    best = [i for i in range(8) if off[i] == min(off)]
    return (best[0] if len(best) == 1 else [i for i in best if i % 2 == 0][0]) + (8 if np.signbit(v) else 0)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -126, 1e-30, 1e30])
def test_codes_are_the_nearest(scale):
    rng = np.random.default_rng(0)
    v = np.float32(rng.standard_normal((3, 70)) * scale).astype(np.float64)
    v[0, :9] = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.25]) * 2.0 ** np.floor(np.log2(scale))
    v[1, 32:64] = 0
    code, byte = ref.quantise(v)
    assert code.shape == (3, 96) and byte.shape == (3, 3) and np.all(code[:, 70:] == 0)
    for n in range(3):
        for j in range(3):
            block = v[n, 32 * j:32 * j + 32]
            m = np.abs(block).max()
            e = -127 if m == 0 else max(int(np.floor(np.log2(m))) - 2, -127)
            assert byte[n, j] == e + 127
            assert [nearest(x, e) for x in block] == list(code[n, 32 * j:32 * j + len(block)])
    # what the codes stand for is off by half a step of the largest binade, or by what passes 6
    d = np.abs(ref.decode(code, byte, 70) - v)
    step = 2.0 ** (np.repeat(byte.astype(np.int64), 32, axis=1)[:, :70] - 127)
    assert np.all(d <= np.maximum(step, np.abs(v) - 6 * step))


def test_ties_go_to_the_even_code_and_the_rest_saturates():
    v = np.zeros((1, 32))
    v[0, :9] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9]
    code, byte = ref.quantise(v)
    assert byte[0, 0] == 127 and list(code[0, :9]) == [6, 0, 2, 2, 4, 4, 6, 6, 7]
    assert list(ref.decode(code, byte, 9)[0]) == [4, 0, 1, 1, 2, 2, 4, 4, 6]


def test_blocks_that_are_not_finite():
    v = np.ones((1, 96))
    v[0, 3], v[0, 70] = np.inf, np.nan
    code, byte = ref.quantise(v)
    assert list(byte[0]) == [255, 125, 255] and np.all(code[0, :32] == 0) and np.all(code[0, 64:] == 0)
    assert np.all(np.isnan(ref.decode(code, byte, 96)[0, :32])) and np.all(ref.decode(code, byte, 96)[0, 32:64] == 1)


def test_values_of_the_grid_are_kept():
    rng = np.random.default_rng(1)
    code = rng.integers(0, 16, size=(4, 64), dtype=np.uint8)
    code[:, ::32] = 7                                   # (a block's largest is 6)
    byte = rng.integers(1, 250, size=(4, 2)).astype(np.uint8)
    v = ref.decode(code, byte, 64)
    assert np.array_equal(ref.decode(*ref.quantise(v), 64), v) and np.array_equal(ref.quantise(v)[1], byte)
    assert np.array_equal(ref.unpack(ref.pack(code)), code)


@pytest.mark.parametrize("rows,K", [(1, 1), (16, 256), (17, 257), (40, 1000)])
def test_places_of_the_scales(rows, K):
    p = ref.scale_places(rows, K)
    assert len(set(p.ravel())) == p.size and p.min() >= 0 and p.max() < -(-rows // 16) * -(-K // 256) * 128
    # lane (g, r) of the instruction: block g of row r in byte 0 of its two, block g + 4 in byte 1
    for r in range(min(rows, 16)):
        for g in range(4):
            assert p[r, g] == 2 * (4 * r + g) and p[r, g + 4] == 2 * (4 * r + g) + 1


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotations(interleaved):
    """They keep lengths, add up, and leave products of queries and keys to the distance."""
    rng = np.random.default_rng(2)
    x, y = rng.standard_normal((2, 5, 2, 20))
    freq = 0.7 ** np.arange(8)
    pos = np.array([0, 1, 5, -3, 1000])

    def rot(v, p):
        return ref.norm_rope(v, p, freq, norm=False, interleaved=interleaved)
    assert np.array_equal(rot(x, pos)[0], x[0]) and np.array_equal(rot(x, pos)[:, :, 16:], x[:, :, 16:])
    assert np.allclose(np.linalg.norm(rot(x, pos), axis=2), np.linalg.norm(x, axis=2), rtol=1e-12)
    assert np.allclose(rot(rot(x, pos), pos + 2), rot(x, 2 * pos + 2), atol=1e-12)
    assert np.allclose((rot(x, pos) * rot(y, pos + 3)).sum(2), (rot(x, 0 * pos) * rot(y, 0 * pos + 3)).sum(2), atol=1e-12)
    one = np.zeros((1, 1, 4))
    one[0, 0, 0] = 1.0
    got = ref.norm_rope(one, [1], [np.pi / 2, 0.0], norm=False, interleaved=interleaved)[0, 0]
    assert np.allclose(got, np.eye(4)[1 if interleaved else 2], atol=1e-15)


def test_norms():
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal((3, 4, 32)), rng.standard_normal(32)
    plain = ref.norm_rope(x, np.zeros(3), np.zeros(0), eps=1e-30)
    assert np.allclose((plain ** 2).mean(2), 1.0, rtol=1e-12)
    assert np.allclose(ref.norm_rope(x, np.zeros(3), np.zeros(0), w, eps=1e-30), plain * w)
    assert np.allclose(ref.norm_rope(x, np.zeros(3), np.zeros(0), w, one_plus=True, eps=1e-30), plain * (1 + w))
    assert np.all(ref.norm_rope(0 * x, np.zeros(3), np.zeros(0)) == 0)
