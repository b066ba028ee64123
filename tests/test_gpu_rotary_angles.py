"""The cosines and sines of rotary positions, as the rows (1, 0) show them."""

import numpy as np
import pytest

from equivariant_gnn_message_amd import e3conv as E

from ._gpu import say
from .test_gpu_attention import host
from .test_gpu_rotary import places

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("layout", ["adjacent", "halves"])
@pytest.mark.parametrize("pairs", [3, 32])
@pytest.mark.parametrize("box", [1.0, 50.0, 1e5])
def test_cosines_and_sines(layout, pairs, box):
    """Within 1.5 u: the result's own rounding, u / 2, and roundings of terms of at most 0.31 that are added last: of
    their last product, its factors and y = x^2 in it, at most 0.25 + 0.15 + 0.31 u.  Relative to a value near zero, x or 1 - 0.29,
    2 u.  The angle is a sum of products in 64 bits, here and there: off by a few roundings of 2^-53, 2^-50 of its terms
    in all."""
    import torch
    n = 4001
    positions, waves = places(pairs, n, pairs, 3, box)
    x = torch.zeros(n, 1, 2 * pairs, device="cuda")
    x[..., 0::2 if layout == "adjacent" else 1] = 1
    if layout == "halves":
        x[..., pairs:] = 0
    got = host(E.e3conv_rotary(x, positions, waves, layout))[:, 0]
    c, s = (got[:, 0::2], got[:, 1::2]) if layout == "adjacent" else (got[:, :pairs], got[:, pairs:])
    p, w = host(positions), host(waves)
    angle, terms = (p[:, None] * w).sum(2), np.abs(p[:, None] * w).sum(2)
    worst = 0.0
    for a, b in ((c, np.cos(angle)), (s, np.sin(angle))):
        off = np.abs(a - b)
        worst = max(worst, float(np.max((off - 2.0 ** -50 * terms) / np.minimum(1.5 * U, 2 * U * np.abs(b)))))
    say(f"[rotary] box {box}, {pairs} pairs {layout}: {worst:.2f} of the bound")
    assert worst <= 1.0
