"""A transformer block with positions in its attention, on the scalars of the convolution.

On the gate-points workload (64 graphs of 64 nodes, 32x0e+32x1o) one forward and backward is

    conv    Plan.forward: messages from the neighbours within the cutoff,
    norm    RMSNormFunction: total = node scalars + the convolution's scalar (l = 0) channels, and its norm,
    turn    RotaryFunction: queries and keys of both maps, as one strided part of the projection, turned by the
            nodes' positions along learned wave vectors (their products then depend on differences of positions: a
            translation of a graph changes nothing, a rotation does, so the block is not rotation invariant),
    attend  DiffAttentionFunction: every node of a graph to every other, two heads of two maps each, with a learned
            weight of the second map,
    heads   RMSNormFunction: each head's result by itself, one weight for all heads,
    out     total + projection of the heads,

with the gradients of all weights and of the positions (the part of the forces that comes through the attention) by
the library's reverse kernels.

Usage: python examples/differential_block.py
"""

import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from equivariant_gnn_message_amd import e3conv as E  # noqa: E402
from equivariant_gnn_message_amd import synth  # noqa: E402

HEADS, DIM, PAIRS, EPS = 2, 8, 3, 1e-5       # of each head: two maps of DIM, values of 2 DIM


def setup(seed=0):
    """The convolution's scalars and the graphs' offsets, and the leaves of the autograd graph."""
    import torch
    inp = synth.make_inputs(1)
    w = inp.workload
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    plan = E.Plan(w.irreps_in, w.lmax, w.irreps_out, w.avg_num_neighbors)
    row_ptr = E.e3conv_csr_from_receivers(t(inp.receivers.astype(np.int32)), inp.num_nodes)
    x = t(inp.x)
    conv = plan.forward(x, t(inp.y), t(inp.s), t(inp.senders.astype(np.int32)), row_ptr)
    data = {"x": x[:, 0, :], "conv": conv[:, 0, :],             # component 0 of (N, num, C): strided rows
            "ptr": torch.arange(w.num_graphs + 1, dtype=torch.int32, device="cuda") * (inp.num_nodes // w.num_graphs)}
    gen = torch.Generator().manual_seed(seed)
    c, inner = plan.channels, 2 * HEADS * DIM
    leaf = lambda *shape, scale=1.0: (scale * torch.randn(shape, generator=gen)).cuda().requires_grad_()
    params = {"norm": torch.ones(c, device="cuda", requires_grad=True), "qkv": leaf(c, 3 * inner, scale=c ** -0.5),
              "waves": leaf(PAIRS, 3), "lam": leaf(HEADS, scale=0.5),
              "head": torch.ones(2 * DIM, device="cuda", requires_grad=True), "out": leaf(inner, c, scale=inner ** -0.5),
              "positions": t(inp.extra["pos"].astype(np.float32)).requires_grad_()}
    return data, params


def block(data, params):
    """Node scalars (N, C)."""
    import torch
    y, total = E.RMSNormFunction.apply(data["conv"], params["norm"], 1, EPS, data["x"])
    n, inner = len(y), 2 * HEADS * DIM
    qkv = y @ params["qkv"]
    qk = E.RotaryFunction.apply(qkv[:, :2 * inner].unflatten(1, (4 * HEADS, DIM)), params["positions"], params["waves"])
    v = qkv[:, 2 * inner:].unflatten(1, (HEADS, 2 * DIM))
    att = E.DiffAttentionFunction.apply(qk[:, :2 * HEADS], qk[:, 2 * HEADS:], v, torch.sigmoid(params["lam"]),
                                        data["ptr"], data["ptr"])
    heads = E.RMSNormFunction.apply(att.reshape(n, inner), params["head"], HEADS, EPS)
    return total + heads @ params["out"]


if __name__ == "__main__":
    import torch
    data, params = setup()
    nodes = block(data, params)
    grads = torch.autograd.grad((nodes ** 2).mean(), list(params.values()))
    print("nodes", tuple(nodes.shape), "rms", f"{nodes.pow(2).mean().sqrt().item():.4f}")
    for name, g in zip(params, grads):
        print(f"gradient of {name:9s} {tuple(g.shape)}, rms {g.pow(2).mean().sqrt().item():.3e}", flush=True)
