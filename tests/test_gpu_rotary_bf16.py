"""Rotary positions in bf16: products of turned rows depend on differences of positions."""

import pytest

from equivariant_gnn_message_amd import e3conv as E

from ._gpu import say
from .test_gpu_rotary import draw, places

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["adjacent", "halves"])
def test_products_depend_on_differences(layout):
    """All positions moved by one vector.  Each turned element is off by 11 u of its pair's size and by its rounding
    of 2^-8, so a product of two rows by twice that of their lengths' product and its square; there are two products."""
    import torch
    q, k = draw(1, "bf16", 50, 2, 32), draw(2, "bf16", 50, 2, 32)
    positions, waves = places(3, 50, 16, 3)
    positions = torch.round(positions * 8) / 8                # sums with the vector are exact
    move = torch.tensor([16.0, -32.0, 64.0], device="cuda")
    turned = lambda t, p: E.e3conv_rotary(t, p, waves, layout).double()
    dot = lambda p: (turned(q, p) * turned(k, p.flip(0))).sum(2)
    off = (dot(positions) - dot(positions + move)).abs() / (q.double().norm(dim=2) * k.double().norm(dim=2))
    each = 2.0 ** -8 + 11 * 2.0 ** -24
    say(f"[rotary] bf16 moved: {float(off.max()):.2e}")
    assert 0 < float(off.max()) <= 2 * (2 * each + each ** 2)
