"""The exact 4-bit data shows what a kernel may do wrong (host only): nothing that is left out or scaled by another
block's scale passes for the product."""
import numpy as np
import pytest

from oracle import mx4_ref as ref
from tests.mx4_exact import pair, product

K = 1 << 20


@pytest.mark.parametrize("K", [K, K - 33])
def test_what_is_left_out_shows(K):
    q, w = pair(3, 3, 40, K, 3)
    want = product(q, w).numpy()
    assert np.mean(want == 0) < 0.01                            # zero outputs do not pass
    step = 512
    cut = lambda a, b: q.values[:, a:b] @ w.values[:, a:b].T    # noqa: E731
    # the last part of 2 to 16, the first and the last step, the last block: nearly every output changes
    for a, b in [(K - K // n, K) for n in (2, 4, 16)] + [(0, step), (K - step, K), (K // step * step - step, K // step * step)]:
        assert np.mean(cut(a, b) == 0) < 0.05
    assert np.mean(cut(K - K % 32 if K % 32 else K - 32, K) == 0) < 0.2


def test_scales_of_another_block_show():
    q, w = pair(4, 2, 20, 1 << 16, 3)
    want = product(q, w).numpy()
    factor = np.ldexp(1.0, (w.bytes.astype(int) - np.roll(w.bytes, 1, axis=1).astype(int))[0]).repeat(32)
    for blocks in (8, 512):                                     # of the last ones
        f = np.where(np.arange(1 << 16) < (1 << 16) - 32 * blocks, 1.0, factor)
        assert np.mean((q.values * f) @ w.values.T == want) < 0.05


def test_the_data_is_what_it_says():
    q, w = pair(5, 3, 4, 1000, 127)
    for s in (q, w):
        v = ref.decode(ref.unpack(s.packed), s.bytes, 1000)
        assert np.array_equal(v, s.values * np.ldexp(1.0, s.bytes.astype(int) - 127).repeat(32, axis=1)[:, :1000])
    assert np.all(q.bytes[0].astype(int) + w.bytes[0] == 254)
    # rows that lq_mx4_quant_rows makes of the values: the scales are the blocks' own
    q, _ = pair(6, 3, 4, 1000, 127, low=-125, top=True)
    x = ref.decode(ref.unpack(q.packed), q.bytes, 1000)
    code, scale = ref.quantise(x)
    assert np.array_equal(scale, q.bytes)
    assert np.array_equal(x, x.astype(np.float32)) and np.array_equal(ref.decode(code, scale, 1000), x)
