"""Root-mean-square norm, rotary positions and differential attention as they are used together: the example block
against the fp64 oracles chained by hand, and the three in one stream and one captured graph with padded bf16 batches."""

import os
import sys

import numpy as np
import pytest

from oracle import diff_attention, rms, rotary
from equivariant_gnn_message_amd import e3conv as E

from ._gpu import say
from .test_gpu_attention import dev, host, ptr

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_block_equals_chained_oracles():
    """fp32, six operators deep: each is within 1e-5 of its result's RMS (the bar of the convolution), and the
    gradients pass them all, so 1e-4 of the RMS holds with room.  The angles add their own: positions of 32 bits
    times waves are exact to 2^-24 of up to some tens of radians, 1e-6."""
    import torch
    import differential_block as G
    data, params = G.setup()
    nodes = G.block(data, params)
    gen = torch.Generator().manual_seed(9)
    grad = torch.randn(nodes.shape, generator=gen).cuda()
    got = dict(zip(params, torch.autograd.grad(nodes, list(params.values()), grad)))
    torch.cuda.synchronize()
    w = {name: host(t.detach()) for name, t in params.items()}
    conv, x, p = host(data["conv"]), host(data["x"]), data["ptr"].cpu().numpy()
    eps, n, heads, dim = float(np.float32(G.EPS)), len(conv), G.HEADS, G.DIM
    inner = 2 * heads * dim
    # values
    first = rms.rms_norm(conv, 1, w["norm"], eps, x)[0]
    qkv = first["y"] @ w["qkv"]
    qk0, v = qkv[:, :2 * inner].reshape(n, 4 * heads, dim), qkv[:, 2 * inner:].reshape(n, heads, 2 * dim)
    qk = rotary.rotary(qk0, w["positions"], w["waves"])[0]
    lam = 1 / (1 + np.exp(-w["lam"]))
    args = (qk[:, :2 * heads], qk[:, 2 * heads:], v, lam, p, p, float(np.float32(dim ** -0.5)))
    att = diff_attention.diff_attention(*args)["out"].reshape(n, inner)
    last = rms.rms_norm(att, heads, w["head"], eps)[0]
    want = first["total"] + last["y"] @ w["out"]
    # gradients, from the result back
    g = host(grad)
    b3 = rms.rms_norm_backward(att, heads, w["head"], last["rstd"], g @ w["out"].T)[0]
    b2 = diff_attention.diff_attention(*args, grad=b3["dx"].reshape(n, heads, 2 * dim))
    b1 = rotary.rotary_backward(qk0, w["positions"], w["waves"], np.concatenate([b2["dq"], b2["dk"]], 1))[0]
    g_qkv = np.concatenate([b1["dx"].reshape(n, 2 * inner), b2["dv"].reshape(n, inner)], 1)
    b0 = rms.rms_norm_backward(first["total"], 1, w["norm"], first["rstd"], g_qkv @ w["qkv"].T, g)[0]
    ref = {"norm": b0["dw"], "qkv": first["y"].T @ g_qkv, "waves": b1["dw"], "lam": b2["dlam"] * lam * (1 - lam),
           "head": b3["dw"], "out": last["y"].T @ g, "positions": b1["dp"]}
    for name, a, b in [("nodes", nodes, want)] + [(k, got[k], ref[k]) for k in ref]:
        err = float(np.abs(host(a.detach()) - b).max() / np.sqrt((b ** 2).mean()))
        say(f"[differential block] {name}: max err / RMS {err:.2e}")
        assert err <= 1e-4, (name, err)


def chain(t, masks):
    """The three operators and their reverse passes, back to back; all results."""
    y, total, rstd = E.e3conv_rms_norm(t["x"], t["w"], 1, 1e-5, t["r"], masks)
    qk, v = y[:, :8 * 32].unflatten(1, (8, 32)), y[:, 8 * 32:].unflatten(1, (2, 64))
    turned = E.e3conv_rotary(qk, t["pos"], t["waves"], "halves", masks)
    out, second, lse = E.e3conv_diff_attention(turned[:, :4], turned[:, 4:], v, t["lam"], t["p"], t["p"], None, masks, masks)
    z, _, rz = E.e3conv_rms_norm(out.reshape(len(y), 128), t["hw"], 2, 1e-5, None, masks)
    gz, ghw = E.e3conv_rms_norm_backward(out.reshape(len(y), 128), t["hw"], 2, rz, t["g"], None, masks)
    gq, gk, gv, glam = E.e3conv_diff_attention_backward(turned[:, :4], turned[:, 4:], v, t["lam"], out, second, lse,
                                                        gz.view_as(out), t["p"], t["p"], None, masks, masks)
    import torch
    gqk, gp, gwaves = E.e3conv_rotary_backward(qk, t["pos"], t["waves"], torch.cat([gq, gk], 1), "halves", masks)
    gy = torch.cat([gqk.flatten(1), gv.flatten(1)], 1)
    gx, gw = E.e3conv_rms_norm_backward(total, t["w"], 1, rstd, gy, None, masks)
    return [y, total, turned, out, z, ghw, gq, gk, gv, glam, gqk, gp, gwaves, gx, gw]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_together_captured_and_on_two_streams(dtype):
    """A padded ragged batch whose padding holds NaN: results are finite and 0 there, and a captured run, replayed
    between eager ones, and runs on two streams at once give the eager run's bits."""
    import torch
    t_ = torch.bfloat16 if dtype == "bf16" else torch.float32
    lens = [70, 0, 33, 1, 300, 64]
    n, gen = sum(lens), torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=gen)
    mask = (torch.rand(n, generator=gen) < 0.8).cuda()
    t = {"x": r(n, 384).to(t_), "r": r(n, 384).to(t_), "g": r(n, 128).to(t_), "w": r(384), "hw": r(64), "pos": r(n, 3),
         "waves": r(16, 3), "lam": r(2)}
    t = {k: v.cuda() for k, v in t.items()}
    t["p"] = dev(ptr(lens))
    for name in ("x", "r", "g", "pos"):
        t[name][~mask] = float("nan")
    want = [v.clone() for v in chain(t, mask)]
    torch.cuda.synchronize()
    for i, v in enumerate(want):
        assert bool(torch.isfinite(v).all()), i
        if len(v) == n and i < 14:
            assert bool((v[~mask] == 0).all()), i
    same = lambda got: all(torch.equal(a, b) for a, b in zip(got, want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(chain(t, mask))
    torch.cuda.synchronize()
    assert same(got[0]) and same(got[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = chain(t, mask)
    for _ in range(3):
        for v in kept:
            v.zero_()
        graph.replay()
        eager = chain(t, mask)
        torch.cuda.synchronize()
        assert same(kept) and same(eager)
