"""A graph-transformer block next to the convolution, trained for a few steps.

On the gate-points workload (64 graphs of 64 nodes, 32x0e+32x1o) one step is

    conv   E3ConvFunction: messages from the neighbours within the cutoff,
    norm   GroupNormFunction: the scalar (l = 0) channels of its output, per graph, with SiLU,
    attend AttentionFunction: every node of a graph to every other, two heads of 16,
    out    node scalars + attention, and one learned token per graph that pools its nodes
           (queries of another length than the keys),

with the gradients of the weights and of the edge scalars by the library's reverse kernels.

Usage: python examples/graph_block.py [steps]
"""

import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from equivariant_gnn_message_amd import e3conv as E  # noqa: E402
from equivariant_gnn_message_amd import synth  # noqa: E402

HEADS, GROUPS = 2, 8


def setup(seed=0):
    """The plan, the graph, its features, and the weights (leaves of the autograd graph)."""
    import torch
    inp = synth.make_inputs(1)
    w = inp.workload
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    plan = E.Plan(w.irreps_in, w.lmax, w.irreps_out, w.avg_num_neighbors)
    graphs = w.num_graphs
    row_ptr = E.e3conv_csr_from_receivers(t(inp.receivers.astype(np.int32)), inp.num_nodes)
    data = {"x": t(inp.x), "y": t(inp.y), "src": t(inp.senders.astype(np.int32)), "row_ptr": row_ptr,
            "ptr": torch.arange(graphs + 1, dtype=torch.int32, device="cuda") * (inp.num_nodes // graphs),
            "one": torch.arange(graphs + 1, dtype=torch.int32, device="cuda")}
    gen = torch.Generator().manual_seed(seed)
    c = plan.channels
    leaf = lambda *shape, scale=1.0: (scale * torch.randn(shape, generator=gen)).cuda().requires_grad_()
    params = {"s": t(inp.s).requires_grad_(), "weight": torch.ones(c, device="cuda", requires_grad=True),
              "bias": torch.zeros(c, device="cuda", requires_grad=True), "qkv": leaf(c, 3 * c, scale=c ** -0.5),
              "token": leaf(1, HEADS, c // HEADS)}
    target = torch.randn((graphs, c), generator=gen).cuda()
    return plan, data, params, target


def block(plan, data, params):
    """(node scalars (N, C), pooled rows (graphs, C))."""
    import torch
    conv = E.E3ConvFunction.apply(plan, data["x"], data["y"], params["s"], data["src"], data["row_ptr"])
    n, _, c = conv.shape
    # component 0 of (N, num_out, C): strided rows, normalised where they lie
    h = E.GroupNormFunction.apply(conv[:, 0, :], data["ptr"], GROUPS, params["weight"], params["bias"], 1e-5, "silu")
    qkv = (h @ params["qkv"]).view(n, 3 * HEADS, c // HEADS)      # one projection, heads side by side
    q, k, v = qkv[:, :HEADS], qkv[:, HEADS:2 * HEADS], qkv[:, 2 * HEADS:]
    nodes = h + E.AttentionFunction.apply(q, k, v, data["ptr"], data["ptr"]).reshape(n, c)
    graphs = data["one"].numel() - 1
    token = params["token"].expand(graphs, HEADS, c // HEADS)     # the same query row for every graph
    pooled = E.AttentionFunction.apply(token, k, nodes.view(n, HEADS, c // HEADS), data["one"], data["ptr"])
    return nodes, pooled.reshape(graphs, c)


def train(steps=10, rate=0.5, seed=0):
    """Plain gradient descent on the pooled rows; the losses."""
    import torch
    plan, data, params, target = setup(seed)
    losses = []
    for _ in range(steps):
        _, pooled = block(plan, data, params)
        loss = ((pooled - target) ** 2).mean()
        grads = torch.autograd.grad(loss, list(params.values()))
        with torch.no_grad():
            for p, g in zip(params.values(), grads):
                p -= rate * g
        losses.append(loss.item())
    return losses


if __name__ == "__main__":
    for i, loss in enumerate(train(int(sys.argv[1]) if len(sys.argv) > 1 else 10)):
        print(f"step {i}: loss {loss:.5f}", flush=True)
