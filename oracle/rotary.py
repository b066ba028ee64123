"""Oracle for rotary positions over several axes (test infrastructure, fp64).

Pair p of every head of row i is the complex number u + i v and is multiplied by exp(i angle[i, p]),
angle = positions waves^T; the derivative of <g, out> turns g's pairs back, and with d_angle the sum over heads of
u gv - v gu gives d_angle waves for the positions and d_angle^T positions for the waves.  Masked rows give zeros.
"""

import numpy as np


def split(t, pairs, layout):
    """(u, v, rest) views."""
    if layout == "halves":
        return t[..., :pairs], t[..., pairs:2 * pairs], t[..., 2 * pairs:]
    return t[..., 0:2 * pairs:2], t[..., 1:2 * pairs:2], t[..., 2 * pairs:]


def _kept(t, mask):
    t = np.array(t, dtype=np.float64)
    if mask is not None:
        t[np.asarray(mask) == 0] = 0
    return t


def _turn(t, z, pairs, layout):
    out = t.copy()
    u, v, _ = split(t, pairs, layout)
    a, b, _ = split(out, pairs, layout)
    w = (u + 1j * v) * z[:, None]
    a[...], b[...] = w.real, w.imag
    return out


def _sizes(t, pairs, layout):
    """|u| + |v| in both places of each pair, 0 elsewhere."""
    out = np.zeros_like(t)
    u, v, _ = split(t, pairs, layout)
    a, b, _ = split(out, pairs, layout)
    a[...] = b[...] = np.abs(u) + np.abs(v)
    return out


def rotary(x, positions, waves, layout="adjacent", mask=None, u=0.0, r=0.0, sign=1.0):
    """(value, bound) of out: with cosines and sines off by 8 u at most (the rounding of the fraction of a turn, half
    a turn at most, and two units of the function's last place), and results rounded by r."""
    x, positions = _kept(x, mask), _kept(positions, mask)
    waves = np.asarray(waves, dtype=np.float64)
    out = _turn(x, np.exp(1j * sign * (positions @ waves.T)), len(waves), layout)
    e = 11 * u * _sizes(x, len(waves), layout)
    return out, e + r * (np.abs(out) + e)


def rotary_backward(x, positions, waves, g, layout="adjacent", mask=None, u=0.0, r=0.0):
    """(values, bounds): dicts with dx, dp, dw."""
    x, positions, g = (_kept(t, mask) for t in (x, positions, g))
    waves = np.asarray(waves, dtype=np.float64)
    n = len(waves)
    dx, _ = rotary(g, positions, waves, layout, None, 0.0, 0.0, -1.0)
    e = 11 * u * _sizes(g, n, layout)
    a, b, _ = split(x, n, layout)
    gu, gv, _ = split(dx, n, layout)
    eu, ev, _ = split(e, n, layout)
    d = (a * gv - b * gu).sum(1)
    size = (np.abs(a * gv) + np.abs(b * gu)).sum(1)
    e_d = (np.abs(a) * ev + np.abs(b) * eu).sum(1) + (4 * np.sqrt(x.shape[1]) + 3) * u * size
    dp, dw = d @ waves, d.T @ positions
    return ({"dx": dx, "dp": dp, "dw": dw},
            {"dx": e + r * (np.abs(dx) + e),
             "dp": e_d @ np.abs(waves) + (4 * np.sqrt(n) + 2) * u * (np.abs(d) @ np.abs(waves)),
             "dw": e_d.T @ np.abs(positions) + 2 * u * np.abs(dw)})
