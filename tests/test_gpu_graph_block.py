"""The example block (convolution, group norm with SiLU, attention, pooling) as one autograd graph:
its value and gradients against the fp64 oracles chained by hand, and a few steps of training."""

import os
import sys

import numpy as np
import pytest

from oracle import attention, norm

from ._gpu import say

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_block_equals_chained_oracles():
    """fp32 throughout, five operators deep: each is within 1e-5 of its result's RMS (the bar of the
    convolution), and the gradients pass them all, so 1e-4 of the RMS holds with room."""
    import torch
    import graph_block as G
    plan, data, params, target = G.setup()
    with torch.no_grad():
        conv = plan.forward(data["x"], data["y"], params["s"].detach(), data["src"], data["row_ptr"])
    host = lambda t: t.detach().double().cpu().numpy()
    x, w, b, mix, token = host(conv[:, 0, :]), host(params["weight"]), host(params["bias"]), host(params["qkv"]), \
        host(params["token"])
    ptr, one = data["ptr"].cpu().numpy(), data["one"].cpu().numpy()
    n, c = x.shape
    graphs, d = len(one) - 1, c // G.HEADS
    nodes, pooled = G.block(plan, data, params)
    loss = ((pooled - target) ** 2).mean()
    got = dict(zip(params, torch.autograd.grad(loss, list(params.values()))))
    torch.cuda.synchronize()
    # values
    h = norm.group_norm(x, ptr, G.GROUPS, w, b, float(np.float32(1e-5)), "silu")[0]["y"]
    qkv = (h @ mix).reshape(n, 3 * G.HEADS, d)
    q, k, v = qkv[:, :G.HEADS], qkv[:, G.HEADS:2 * G.HEADS], qkv[:, 2 * G.HEADS:]
    scale = np.float32(d ** -0.5)
    att = attention.attention(q, k, v, ptr, ptr, scale)["out"]
    rows = h + att.reshape(n, c)
    tok = np.broadcast_to(token, (graphs, G.HEADS, d))
    pool = attention.attention(tok, k, rows.reshape(n, G.HEADS, d), one, ptr, scale)["out"]
    # gradients, from the loss back
    g_pool = 2 * (pool.reshape(graphs, c) - host(target)) / (graphs * c)
    a2 = attention.attention(tok, k, rows.reshape(n, G.HEADS, d), one, ptr, scale, grad=g_pool.reshape(pool.shape))
    g_rows = a2["dv"].reshape(n, c)
    a1 = attention.attention(q, k, v, ptr, ptr, scale, grad=g_rows.reshape(n, G.HEADS, d))
    g_qkv = np.concatenate([a1["dq"], a1["dk"] + a2["dk"], a1["dv"]], 1).reshape(n, 3 * c)
    g_h = g_rows + g_qkv @ mix.T
    back = norm.group_norm(x, ptr, G.GROUPS, w, b, float(np.float32(1e-5)), "silu", grad=g_h)[0]
    want = {"weight": back["dw"], "bias": back["dc"], "qkv": h.T @ g_qkv,
            "token": a2["dq"].sum(0, keepdims=True)}
    for name, ref, val in [("nodes", rows, nodes), ("pooled", pool.reshape(graphs, c), pooled)] + [
            (k_, want[k_], got[k_]) for k_ in want]:
        err = float(np.abs(host(val) - ref).max() / np.sqrt((ref ** 2).mean()))
        say(f"[block] {name}: max err / RMS {err:.2e}")
        assert err <= 1e-4, (name, err)
    assert bool(torch.isfinite(got["s"]).all()) and bool((got["s"] != 0).any())


def test_training_goes_down():
    import graph_block as G
    losses = G.train(8)
    say("[block] losses", " ".join(f"{v:.4f}" for v in losses))
    assert all(np.isfinite(losses)) and losses[-1] < losses[0]
