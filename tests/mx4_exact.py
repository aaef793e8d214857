"""4-bit rows and weights whose products fp32 sums exactly, whatever the order.

Values are among 0, 0.5, 1, 1.5, 2 and their negatives (some rows: a 4 in every block), scales of both sides
cancel block by block: block j has 2^a_j on one side and 2^-a_j on the other, a_j as wide as asked. Products are
multiples of 1/4, and where the sum of their magnitudes stays below 2^22 every partial sum has 24 bits. So outputs
are compared for equality, and a block, step or part that is left out, read twice or scaled by another's scale
shows."""
import numpy as np
import torch

from oracle import mx4_ref as ref


class Side:
    """One side's codes and scales, with garbage past K and NaN in the scales of rows and blocks that are none."""

    def __init__(self, rng, rows, K, exponents, top=False):
        nb = -(-K // 32)
        self.rows, self.K = rows, K
        mag = rng.integers(0, 5, size=(rows, 32 * nb), dtype=np.uint8)                  # codes of 0 to 2
        if top:
            mag[:, rng.integers(0, 32, nb) + 32 * np.arange(nb)] = 6                    # 4: the scale of the block is its own
            mag[:, 32 * (nb - 1) + (K - 1) % 32] = 6
        code = mag | rng.integers(0, 2, size=mag.shape, dtype=np.uint8) << 3
        code[:, K:] = rng.integers(0, 16, size=(rows, 32 * nb - K), dtype=np.uint8)
        self.values = (ref.GRID[code & 7] * np.where(code & 8, -1.0, 1.0))[:, :K]       # without their scales
        self.packed = ref.pack(code)
        self.bytes = np.broadcast_to((127 + exponents).astype(np.uint8), (rows, nb))
        self.panels = ref.panels(self.bytes, K, fill=255)

    def on(self, device):
        return torch.from_numpy(self.packed).to(device), torch.from_numpy(self.panels).to(device)


def pair(seed, B, N, K, spread, low=None, top=False):
    """(tokens, weights) with scales that cancel; exponents of the weights from low (-spread) to spread."""
    rng = np.random.default_rng(seed)
    a = rng.integers(-spread if low is None else low, spread + 1, size=-(-K // 32))
    return Side(rng, B, K, -a, top), Side(rng, N, K, a)


def product(q, w, device="cpu"):
    """The exact product; refuses data whose sums fp32 might round."""
    a, b = torch.from_numpy(q.values).to(device), torch.from_numpy(w.values).to(device)
    assert float((a.abs() @ b.abs().T).max()) < 2.0 ** 22
    return a @ b.T
