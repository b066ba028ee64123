"""Oracle for group norm with an activation per graph (test infrastructure, fp64).

Over the counted rows of graph b and the channels of a group,
xhat = (x - mean) / sqrt(var + eps), z = w xhat + c, y = act(z); and the derivative
of <g, y>: dz = g act'(z), dw = sum dz xhat, dc = sum dz, and with dn = dz w
dx = (dn - mean(dn) - xhat mean(dn xhat)) / sqrt(var + eps).
"""

import numpy as np
from scipy.special import erf, expit


def activate(z, act):
    """act(z) and act'(z)."""
    if act == "relu":
        return np.maximum(z, 0.0), (z > 0).astype(np.float64)
    if act == "silu":
        e = expit(z)
        return z * e, e * (1 + z * (1 - e))
    if act == "gelu":
        c = 0.5 * (1 + erf(z / np.sqrt(2.0)))
        return z * c, c + z * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    return z, np.ones_like(z)


def group_norm(x, row_ptr, groups, weight, bias, eps, act, row_mask=None, grad=None, u=0.0, r=0.0):
    """(values, bounds): dicts with y, mean, rstd and, where grad is given, dx, dw, dc.

    bounds: how far an evaluation may be off whose fp32 operations round by u, whose
    sums of n terms err by 4 sqrt(n) u of the terms' magnitudes, and whose stored y and
    dx round by r.
    """
    x = np.asarray(x, dtype=np.float64)
    n, c = x.shape
    graphs = len(row_ptr) - 1
    w = np.ones(c) if weight is None else np.asarray(weight, dtype=np.float64)
    b = np.zeros(c) if bias is None else np.asarray(bias, dtype=np.float64)
    val = {"y": np.zeros_like(x), "mean": np.zeros((graphs, groups)),
           "rstd": np.full((graphs, groups), 1 / np.sqrt(eps))}
    tol = {"y": np.zeros_like(x), "mean": np.zeros((graphs, groups)),
           "rstd": np.full((graphs, groups), 4 * u / np.sqrt(eps))}
    if grad is not None:
        for d in (val, tol):
            d.update(dx=np.zeros_like(x), dw=np.zeros(c), dc=np.zeros(c))
    spread = 0.0
    for g in range(graphs):
        rows = np.arange(row_ptr[g], row_ptr[g + 1])
        if row_mask is not None:
            rows = rows[np.asarray(row_mask)[rows] != 0]
        if not len(rows):
            continue
        xb = x[rows].reshape(len(rows), groups, -1)
        size = xb.shape[0] * xb.shape[2]
        long = 4 * np.sqrt(size)
        mu = xb.mean((0, 2))
        xc = xb - mu[:, None]
        var = (xc * xc).mean((0, 2))
        rs = 1 / np.sqrt(var + eps)
        # the mean is summed about a value of the data: its error is that of the spread, plus
        # its own rounding; the variance is summed about a nearby value
        e_mu = u * (long * np.abs(xc).mean((0, 2)) + 4 * np.abs(mu) + 4 * np.abs(xb).max((0, 2)))
        e_rs = rs * (0.5 * (((long + 8) * u * var) + 4 * u * np.abs(xb).max((0, 2)) * np.abs(xc).mean((0, 2))
                            + e_mu ** 2) * rs * rs + 4 * u)
        val["mean"][g], val["rstd"][g] = mu, rs
        tol["mean"][g], tol["rstd"][g] = e_mu, e_rs
        xh = xc * rs[:, None]
        e_xh = (e_mu * rs)[:, None] + np.abs(xh) * (e_rs / rs)[:, None] + 4 * u * np.abs(xh) \
            + 2 * u * np.abs(xb) * rs[:, None]
        flat = lambda t: t.reshape(len(rows), c)
        z = flat(xh) * w + b
        e_z = flat(e_xh) * np.abs(w) + 2 * u * (np.abs(flat(xh) * w) + np.abs(b))
        y, dy = activate(z, act)
        # |act'| <= 1.13 and |act''| <= 1 for every activation (relu: away from 0)
        e_act = 1.13 * e_z + 8 * u * (np.abs(z) + np.abs(y))
        val["y"][rows] = y
        tol["y"][rows] = e_act + r * (np.abs(y) + e_act)
        if grad is None:
            continue
        gr = np.asarray(grad, dtype=np.float64)[rows]
        dz = gr * dy
        e_dz = np.abs(gr) * (e_z + 8 * u * (1 + np.abs(z)))
        if act in ("none", "relu"):
            e_dz = 4 * u * np.abs(dz)
        val["dc"] += dz.sum(0)
        val["dw"] += (dz * flat(xh)).sum(0)
        tol["dc"] += e_dz.sum(0)
        tol["dw"] += (e_dz * np.abs(flat(xh)) + np.abs(dz) * flat(e_xh)).sum(0)
        spread = spread + np.stack([np.abs(dz).sum(0), np.abs(dz * flat(xh)).sum(0)])
        dn, e_dn = (dz * w).reshape(xb.shape), (e_dz * np.abs(w) + 2 * u * np.abs(dz * w)).reshape(xb.shape)
        m = lambda t: t.mean((0, 2))[:, None]
        dx = (dn - m(dn) - xh * m(dn * xh)) * rs[:, None]
        e_m1 = m(e_dn) + long * u * m(np.abs(dn))
        e_m2 = m(e_dn * np.abs(xh) + np.abs(dn) * e_xh) + (long + 2) * u * m(np.abs(dn * xh))
        e = e_dn + e_m1 + np.abs(xh) * e_m2 + e_xh * np.abs(m(dn * xh)) \
            + 4 * u * (np.abs(dn) + np.abs(m(dn)) + np.abs(xh * m(dn * xh)))
        e = e * rs[:, None] + np.abs(dx) * (e_rs / rs)[:, None]
        val["dx"][rows] = flat(dx)
        tol["dx"][rows] = flat(e) + r * (flat(np.abs(dx) + e))
    if grad is not None and n:
        long = 4 * np.sqrt(n)
        tol["dc"] += (long * u) * (spread[0] if not np.isscalar(spread) else 0.0)
        tol["dw"] += (long * u) * (spread[1] if not np.isscalar(spread) else 0.0)
    return val, tol
