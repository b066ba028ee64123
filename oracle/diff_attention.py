"""Oracle for differential attention among the nodes of each graph (test infrastructure, fp64).

Graph by graph and head by head from the definition, with maps m = 0, 1 (heads 2 h + m of q, 2 c + m of k):

    S_m = scale q_m k_m^T over the graph's unmasked queries and keys,
    P_m = exp(S_m - lse_m), out = (P_0 - lam P_1) v, second = P_1 v,

and the derivative of <g, out>: with dP = g v^T, delta_m = sum_j P_m dP, dS_0 = P_0 (dP - delta_0) and
dS_1 = -lam P_1 (dP - delta_1): dq_m = scale dS_m k_m, dk_m = scale dS_m^T q_m, dv = (P_0 - lam P_1)^T g,
dlam = - the sum of P_1 dP; query heads that share kv head c add up.  A query that sees no key has out = 0,
lse = -inf and no gradient.

``bounds`` derives from the same quantities how far a rounded evaluation may be from these values.
"""

import numpy as np

from .attention import segments


def diff_attention(q, k, v, lam, q_ptr, k_ptr, scale, q_mask=None, k_mask=None, grad=None):
    """dict with out, second, lse and, where grad is given, dq, dk, dv, dlam."""
    return bounds(q, k, v, lam, q_ptr, k_ptr, scale, 0.0, 0.0, q_mask, k_mask, grad)[0]


def bounds(q, k, v, lam, q_ptr, k_ptr, scale, u, r, q_mask=None, k_mask=None, grad=None):
    """(values, elementwise bounds of |computed - exact|) for an evaluation whose fp32 operations round by u,
    whose sums of n terms err by at most 4 sqrt(n) u of their terms' magnitudes (independent roundings), and which
    rounds P_m and P_0 - lam P_1 and dS_m before their products, and every result, by r."""
    q, k, v, lam = (np.asarray(t, dtype=np.float64) for t in (q, k, v, lam))
    nq, h2, d = q.shape
    heads, n = h2 // 2, h2 // k.shape[1]
    val = {"out": np.zeros((nq, heads, v.shape[2])), "second": np.zeros((nq, heads, v.shape[2])),
           "lse": np.full((nq, heads, 2), -np.inf)}
    if grad is not None:
        grad = np.asarray(grad, dtype=np.float64)
        val.update(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v), dlam=np.zeros(heads))
    tol = {name: np.zeros(t.shape) for name, t in val.items()}
    spread = np.zeros(heads)
    for rows, cols in segments(q_ptr, k_ptr, q_mask, k_mask):
        long_k, dims = 4 * np.sqrt(len(cols)), 4 * np.sqrt(max(d, v.shape[2]))
        long_q = 4 * np.sqrt(len(rows) * n)
        for h in range(heads):
            c, w = h // n, abs(lam[h])
            vh = v[cols, c]
            av = np.abs(vh)
            p, ep, o, eo = [], [], [], []
            for m in (0, 1):
                qh, kh = q[rows, 2 * h + m], k[cols, 2 * c + m]
                s = scale * (qh @ kh.T)
                top = s.max(1, keepdims=True)
                lse = top + np.log(np.exp(s - top).sum(1, keepdims=True))
                p.append(np.exp(s - lse))
                val["lse"][rows, h, m] = lse[:, 0]
                # logits: their dot product, the scaling, and exp's argument in units of the largest logit
                es = u * ((dims + 4) * abs(scale) * (np.abs(qh) @ np.abs(kh).T) + 4 * np.abs(s)
                          + 4 * np.abs(s).max(1, keepdims=True) + 8)
                el = (p[m] * es).sum(1, keepdims=True) + (long_k + 4) * u + 2 * u * np.abs(lse)
                tol["lse"][rows, h, m] = el[:, 0]
                ep.append(p[m] * (es + el))                                   # of the probabilities, in fp32
                o.append(p[m] @ vh)
                eo.append((ep[m] + (r + long_k * u) * p[m]) @ av + 2 * u * np.abs(o[m]))
            out = o[0] - lam[h] * o[1]
            e_out = eo[0] + w * eo[1] + 2 * u * w * np.abs(o[1])
            val["out"][rows, h], val["second"][rows, h] = out, o[1]
            tol["out"][rows, h] = e_out + r * (np.abs(out) + e_out)
            tol["second"][rows, h] = eo[1] + r * (np.abs(o[1]) + eo[1])
            if grad is None:
                continue
            gh = grad[rows, h]
            g = np.abs(gh)
            dp = gh @ vh.T
            edp = u * dims * (g @ av.T)
            diff = p[0] - lam[h] * p[1]
            e_diff = ep[0] + w * ep[1] + 2 * u * (p[0] + w * p[1])
            val["dv"][cols, c] += diff.T @ gh
            tol["dv"][cols, c] += (e_diff + (r + (long_q + 4) * u) * np.abs(diff)).T @ g
            # delta_1 from second, delta_0 from out and delta_1, as they are stored
            ed1 = (g * (tol["second"][rows, h] + dims * u * np.abs(o[1]))).sum(1, keepdims=True)
            ed0 = (g * (tol["out"][rows, h] + dims * u * np.abs(out))).sum(1, keepdims=True) + w * ed1
            for m, ed, f in ((0, ed0, 1.0), (1, ed1, -lam[h])):
                delta = (p[m] * dp).sum(1, keepdims=True)
                ds = p[m] * (dp - delta)
                eds = ep[m] * np.abs(dp - delta) + p[m] * (edp + ed + 4 * u * (np.abs(dp) + np.abs(delta)))
                ads = np.abs(ds)
                qh, kh, a = np.abs(q[rows, 2 * h + m]), np.abs(k[cols, 2 * c + m]), abs(scale * f)
                val["dq"][rows, 2 * h + m] = scale * f * (ds @ k[cols, 2 * c + m])
                val["dk"][cols, 2 * c + m] += scale * f * (ds.T @ q[rows, 2 * h + m])
                tol["dq"][rows, 2 * h + m] = a * ((eds + (r + (long_k + 4) * u) * ads) @ kh)
                tol["dk"][cols, 2 * c + m] += a * ((eds + (r + (long_q + 6) * u) * ads).T @ qh)
            # dlam: delta_1 as above plus the sum of the unrounded P_1 (dP - delta_1): the error of delta_1 cancels
            # as far as the P_1 of a row add up to one
            terms = p[1] * np.abs(dp)
            val["dlam"][h] -= (p[1] * dp).sum()
            delta = np.abs((p[1] * dp).sum(1, keepdims=True))
            unit = ep[1].sum(1, keepdims=True) + long_k * u
            tol["dlam"][h] += (ep[1] * np.abs(dp - (p[1] * dp).sum(1, keepdims=True)) + p[1] * edp).sum() \
                + (unit * ed1).sum() + ((long_k + 8) * u * (terms + p[1] * delta)).sum()
            spread[h] += np.abs((p[1] * dp).sum(1)).sum()
    if grad is not None:
        rows_n = max(nq, 1)
        tol["dlam"] += (4 * np.sqrt(rows_n) + 4) * u * spread
        for t in ("dq", "dk", "dv"):
            tol[t] += (r + 4 * u) * np.abs(val[t]) + r * tol[t]
    return val, tol
