"""Oracle for the root-mean-square norm with a residual (test infrastructure, fp64).

s = x + residual; over each group of a row's channels rstd = 1 / sqrt(mean(s^2) + eps) and y = w s rstd,
w[c] = weight[c mod len(weight)]; and the derivative of <g, y> + <gt, s> at given s and rstd:
xhat = s rstd, dn = w g, ds = rstd (dn - xhat mean(dn xhat)) + gt, dw = the sum of g xhat over all that w[j]
multiplies.  Masked rows: y = s = ds = 0, rstd = 1 / sqrt(eps).
"""

import numpy as np


def _kept(t, mask):
    t = np.asarray(t, dtype=np.float64)
    return t if mask is None else np.where(np.asarray(mask, bool)[:, None], t, 0.0)


def _weight(weight, c):
    return np.ones(c) if weight is None else np.tile(np.asarray(weight, dtype=np.float64), c // len(weight))


def rms_norm(x, groups, weight=None, eps=1e-5, residual=None, mask=None, u=0.0, r=0.0):
    """(values, bounds): dicts with y, total, rstd.

    bounds: how far an evaluation may be off whose fp32 operations round by u, whose sums of n
    terms err by 4 sqrt(n) u of the terms' magnitudes, and whose stored y and total round by r.
    """
    s = _kept(x, mask)
    n, c = s.shape
    add = 0.0
    if residual is not None:
        s, add = s + _kept(residual, mask), u
    rows = s.reshape(n, groups, c // groups)
    size = rows.shape[2]
    rstd = 1 / np.sqrt((rows ** 2).mean(2) + eps)
    # the terms are squares: relative errors; half of the mean's goes to the root
    e_rs = 0.5 * ((4 * np.sqrt(size) + 4) * u + 2 * add) + 4 * u
    y = (rows * rstd[..., None]).reshape(n, c) * _weight(weight, c)
    e_y = np.abs(y) * (e_rs + add + 3 * u)
    e_s = np.abs(s) * add
    return ({"y": y, "total": s, "rstd": rstd},
            {"y": e_y + r * (np.abs(y) + e_y), "total": e_s + r * (np.abs(s) + e_s), "rstd": rstd * e_rs})


def rms_norm_backward(s, groups, weight, rstd, g, gt=None, mask=None, u=0.0, r=0.0):
    """(values, bounds): dicts with dx and dw, as above."""
    s, g = _kept(s, mask), _kept(g, mask)
    n, c = s.shape
    size, shape = c // groups, (n, groups, c // groups)
    rstd = np.asarray(rstd, dtype=np.float64)[..., None]
    xh, dn = s.reshape(shape) * rstd, (g * _weight(weight, c)).reshape(shape)
    m = (dn * xh).mean(2, keepdims=True)
    e_m = (4 * np.sqrt(size) + 5) * u * np.abs(dn * xh).mean(2, keepdims=True)
    d = rstd * (dn - xh * m)
    e = rstd * (np.abs(xh) * e_m + 5 * u * (np.abs(dn) + np.abs(xh * m)))
    if gt is not None:
        d = d + _kept(gt, mask).reshape(shape)
        e = e + u * np.abs(d)
    live = np.ones((n, 1, 1)) if mask is None else np.asarray(mask, bool)[:, None, None]
    dx, e = (d * live).reshape(n, c), (e * live).reshape(n, c)
    terms = g.reshape(shape) * xh
    period = c if weight is None else len(weight)
    fold = lambda t: t.reshape(-1, period).sum(0)
    terms_n = max(n * (c // period), 1)
    return ({"dx": dx, "dw": fold(terms)},
            {"dx": e + r * (np.abs(dx) + e), "dw": (4 * np.sqrt(terms_n) + 4) * u * fold(np.abs(terms))})
