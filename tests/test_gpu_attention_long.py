"""Attention over many keys of few kinds (nodes of one species with the same embedding): equal terms round alike,
so the error of a plain running sum grows with their number and not with its root.

The bounds are those of oracle.attention.bounds for one query; all queries are the same, and enough of them to fill
the device, so that the keys are not split.  And calls of more work-groups than one axis of a launch takes.
"""

import numpy as np
import pytest

from oracle import attention
from equivariant_gnn_message_amd import e3conv as E

from ._gpu import say
from .test_gpu_attention import U, dev, dtype_of, host, ptr

pytestmark = pytest.mark.gpu

HEADS, DIM = 4, 32


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("keys", [20000, 100000])
@pytest.mark.parametrize("gap", [5.0625, 3.3125])
def test_logits_of_two_values(dtype, keys, gap):
    """One key in two has a logit lower by `gap` (exact in bf16): probabilities p and p exp(-gap)."""
    import torch
    gen = torch.Generator().manual_seed(keys)
    queries = 256 * (3 if dtype == "f32" else 4) * 128 // HEADS      # one work-group on every place of the device
    q = torch.zeros((queries, HEADS, DIM))
    q[:, :, 0] = 1.0
    k = torch.zeros((keys, HEADS, DIM))
    k[:, :, 0] = -gap * (torch.rand((keys, HEADS), generator=gen) < 0.5)
    v = torch.randn((keys, HEADS, DIM), generator=gen)
    q, k, v = (t.to(dtype_of(dtype)).cuda() for t in (q, k, v))
    args = E.AttentionArgs(dtype=0 if dtype == "f32" else 1, num_graphs=1, heads_q=HEADS, heads_kv=HEADS, dim_qk=DIM,
                           dim_v=DIM, num_q=queries, num_k=keys, scale=1.0)
    assert E.e3conv_attention_workspace_size(args) == 0               # the keys stay unsplit
    say(f"[attention] {dtype} {queries} equal queries, {keys} keys of two kinds")
    out, lse = E.e3conv_attention(q, k, v, dev(ptr([queries])), dev(ptr([keys])), 1.0)
    torch.cuda.synchronize()
    assert bool((lse == lse[:1]).all()) and bool((out == out[:1]).all())
    u, r = U[dtype]
    want, tol = attention.bounds(host(q[:1]), host(k), host(v), [0, 1], [0, keys], 1.0, u, r)
    for name, got in (("lse", lse), ("out", out)):
        off = np.abs(host(got[:1]) - want[name])
        say(f"  {name}: max err {off.max():.3e}, bound {tol[name].min():.3e}")
        assert np.all(off <= tol[name]), name


def test_more_work_groups_than_one_axis_of_a_launch():
    """A million graphs of one node with 64 heads: 69 million work-groups of 64 threads are more than 2^32 threads.
    With one key P = 1, so out = v, lse = scale <q, k>, grad_v = grad_out, and grad_q, grad_k are the rounding of
    dP - delta (each a sum of 8 products, in fp32) times scale k or q."""
    import torch
    graphs, heads, dim = (1 << 20) - 1, 64, 8
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k, v, g = (torch.randn((graphs, heads, dim), generator=gen, device="cuda").bfloat16() for _ in range(4))
    p = torch.arange(graphs + 1, dtype=torch.int32, device="cuda")
    say(f"[attention] bf16 {graphs} graphs of one node, {heads} heads of {dim}")
    out, lse = E.e3conv_attention(q, k, v, p, p, 0.5)
    gq, gk, gv = E.e3conv_attention_backward(q, k, v, out, lse, g, p, p, 0.5)
    torch.cuda.synchronize()
    u = 2.0 ** -24
    assert torch.equal(out, v) and torch.equal(gv, g)
    dot, size = (0.5 * (t.float()).sum(2) for t in (q * k.float(), (q * k.float()).abs()))
    assert bool(((lse - dot).abs() <= 24 * u * (size + 1)).all())
    slack = 24 * u * (g * v.float()).abs().sum(2)[:, :, None] * 0.5
    for got, other in ((gq, k), (gk, q)):
        assert bool((got.float().abs() <= slack * other.float().abs() * (1 + 2.0 ** -8) + 1e-38).all())
