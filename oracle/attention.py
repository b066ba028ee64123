"""Oracle for attention among the nodes of each graph (test infrastructure, fp64).

Graph by graph and head by head from the definition:

    S = scale q k^T over the graph's unmasked queries and keys,
    P = exp(S - lse), lse = log sum_j exp(S_j), out = P v,

and the derivative of <g, out>: with dP = g v^T and dS = P (dP - sum_j P dP),
dq = scale dS k, dk = scale dS^T q, dv = P^T g, where the query heads
h = c n .. c n + n - 1 share kv head c (their contributions to dk and dv add up).
A query that sees no key has out = 0, lse = -inf and no gradient.

``bounds`` derives from the same quantities how far a rounded evaluation may be
from these values.
"""

import numpy as np


def segments(q_ptr, k_ptr, q_mask=None, k_mask=None):
    """(query rows, key rows) of each graph after the masks."""
    for g in range(len(q_ptr) - 1):
        rows, cols = np.arange(q_ptr[g], q_ptr[g + 1]), np.arange(k_ptr[g], k_ptr[g + 1])
        if q_mask is not None:
            rows = rows[np.asarray(q_mask)[rows] != 0]
        if k_mask is not None:
            cols = cols[np.asarray(k_mask)[cols] != 0]
        if len(rows) and len(cols):
            yield rows, cols


def attention(q, k, v, q_ptr, k_ptr, scale, q_mask=None, k_mask=None, grad=None):
    """dict with out, lse and, where grad is given, dq, dk, dv."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    nq, hq, d = q.shape
    n = hq // k.shape[1]
    res = {"out": np.zeros((nq, hq, v.shape[2])), "lse": np.full((nq, hq), -np.inf)}
    if grad is not None:
        grad = np.asarray(grad, dtype=np.float64)
        res.update(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v))
    for rows, cols in segments(q_ptr, k_ptr, q_mask, k_mask):
        for h in range(hq):
            c = h // n
            qh, kh, vh = q[rows, h], k[cols, c], v[cols, c]
            s = scale * (qh @ kh.T)
            top = s.max(1, keepdims=True)
            e = np.exp(s - top)
            total = e.sum(1, keepdims=True)
            p = e / total
            out = p @ vh
            res["out"][rows, h] = out
            res["lse"][rows, h] = (top + np.log(total))[:, 0]
            if grad is not None:
                g = grad[rows, h]
                dp = g @ vh.T
                ds = p * (dp - (p * dp).sum(1, keepdims=True))
                res["dq"][rows, h] = scale * (ds @ kh)
                res["dk"][cols, c] += scale * (ds.T @ qh)
                res["dv"][cols, c] += p.T @ g
    return res


def bounds(q, k, v, q_ptr, k_ptr, scale, u, r, q_mask=None, k_mask=None, grad=None):
    """Elementwise bounds of |computed - exact| for an evaluation whose fp32
    operations round by u, whose sums of n terms err by at most 4 sqrt(n) u
    of their terms' magnitudes (independent roundings), and which rounds P and dS
    before their products, and every result, by r."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    nq, hq, d = q.shape
    n = hq // k.shape[1]
    tol = {"out": np.zeros((nq, hq, v.shape[2])), "lse": np.zeros((nq, hq))}
    if grad is not None:
        grad = np.asarray(grad, dtype=np.float64)
        tol.update(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v))
    exact = attention(q, k, v, q_ptr, k_ptr, scale, q_mask, k_mask, grad)
    for rows, cols in segments(q_ptr, k_ptr, q_mask, k_mask):
        long_k, dims = 4 * np.sqrt(len(cols)), 4 * np.sqrt(max(d, v.shape[2]))
        for h in range(hq):
            c = h // n
            qh, kh, vh = q[rows, h], k[cols, c], v[cols, c]
            s = scale * (qh @ kh.T)
            # logits: their dot product, the scaling, and exp's argument in units of the
            # largest logit (base-2 conversion and subtraction of the maximum)
            es = u * ((dims + 4) * abs(scale) * (np.abs(qh) @ np.abs(kh).T) + 4 * np.abs(s)
                      + 4 * np.abs(s).max(1, keepdims=True) + 8)
            p = np.exp(s - exact["lse"][rows, h][:, None])
            el = (p * es).sum(1, keepdims=True) + (long_k + 4) * u + 2 * u * np.abs(exact["lse"][rows, h])[:, None]
            ep = p * (es + el)                                    # of the probabilities, in fp32
            av = np.abs(vh)
            eo = (ep + (r + long_k * u) * p) @ av
            tol["out"][rows, h] = eo + (r + 2 * u) * np.abs(exact["out"][rows, h])
            tol["lse"][rows, h] = el[:, 0]
            if grad is None:
                continue
            g = np.abs(grad[rows, h])
            long_q = 4 * np.sqrt(len(rows) * n)
            dp = grad[rows, h] @ vh.T
            delta = (p * dp).sum(1, keepdims=True)
            ds = np.abs(p * (dp - delta))
            edp = u * dims * (g @ av.T)
            ed = ((g * (tol["out"][rows, h] + dims * u * np.abs(exact["out"][rows, h]))).sum(1, keepdims=True))
            eds = ep * np.abs(dp - delta) + p * (edp + ed + 4 * u * (np.abs(dp) + np.abs(delta)))
            a = abs(scale)
            tol["dq"][rows, h] = a * ((eds + (r + (long_k + 4) * u) * ds) @ np.abs(kh))
            tol["dk"][cols, c] += a * ((eds + (r + (long_q + 4) * u) * ds).T @ np.abs(qh))
            tol["dv"][cols, c] += (ep + (r + (long_q + 4) * u) * p).T @ g
    for t in ("dq", "dk", "dv"):
        if grad is not None:
            tol[t] += (r + 2 * u) * np.abs(exact[t])
    return exact, tol
