"""Infinities and NaN in rows that count: masked queries keep zero gradients, and the aligned and the
element-by-element path agree."""

import numpy as np
import pytest

from equivariant_gnn_message_amd import e3conv as E

from ._gpu import say
from .test_gpu_attention import dev, draw, host, ptr

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens_q,lens_k", [([40], [70]), ([5], [20011]), ([300], [2000])], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_masked_queries_of_a_graph_with_bad_keys(dtype, lens_q, lens_k, bad):
    """The keys split or not: a masked query has out = 0, lse = -infinity and grad_q = 0, whatever the
    counted keys and values hold."""
    import torch
    q, k, v, g = draw(3, dtype, lens_q, lens_k, 4, 2, 24, 40)
    k[1, 0, 3] = v[2, 1, 5] = v[-1, 0, 0] = bad
    mask = np.arange(sum(lens_q)) % 3 != 1
    p, kp = dev(ptr(lens_q)), dev(ptr(lens_k))
    say(f"[attention] {dtype} {lens_q} queries, {lens_k} keys, {bad} among them")
    out, lse = E.e3conv_attention(q, k, v, p, kp, q_mask=dev(mask))
    gq, _, _ = E.e3conv_attention_backward(q, k, v, out, lse, g, p, kp, q_mask=dev(mask))
    torch.cuda.synchronize()
    hole = dev(~mask)
    assert not out[hole].any() and bool(torch.isneginf(lse[hole]).all())
    assert not gq[hole].any()


@pytest.mark.parametrize("dim", [8, 24, 40, 48, 72, 96, 104])
@pytest.mark.parametrize("lens", [[50], [9, 300], [3000]], ids=str)
def test_infinite_key_aligned_or_not(dim, lens):
    """bf16, an infinity in a key that gives every query a logit of -infinity: the key has no weight, and rows
    loaded by whole units and element by element give the same bits."""
    import torch
    q, k, v, g = draw(4, "bf16", lens, lens, 2, 2, dim, dim)
    q[:, :, 0] = -q[:, :, 0].abs() - 0.5
    k[lens[0] - 1, :, 0] = float("inf")
    p = dev(ptr(lens))
    say(f"[attention] bf16 {lens} nodes, {dim} dimensions, an infinite key")

    def shifted(t):
        return torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)

    mask = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
    out, lse = E.e3conv_attention(q, k, v, p, p)
    ref, lse_ref = E.e3conv_attention(shifted(q), shifted(k), shifted(v), p, p)
    mask[lens[0] - 1] = False
    k_finite = torch.where(mask[:, None, None], k, 0)
    without, _ = E.e3conv_attention(q, k_finite, v, p, p, k_mask=mask)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out).all()) and torch.equal(out, ref) and torch.equal(lse, lse_ref)
    assert torch.equal(out, without)
    grads = E.e3conv_attention_backward(q, k, v, out, lse, g, p, p)
    refs = E.e3conv_attention_backward(shifted(q), shifted(k), shifted(v), out, lse, g, p, p)
    torch.cuda.synchronize()
    for a, b in zip(grads, refs):
        assert np.array_equal(host(a), host(b), equal_nan=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [24, 33, 64])
@pytest.mark.parametrize("lens", [[40, 50, 60], [2000, 333, 1000]], ids=str)
def test_bad_values_stay_in_their_graph(dtype, dim, lens):
    """Infinities and NaN in the counted rows of one graph change no bit of the others."""
    import torch
    p = dev(ptr(lens))
    q, k, v, g = draw(9, dtype, lens, lens, 4, 2, dim, dim)
    say(f"[attention] {dtype} {lens} nodes, {dim} dimensions, bad values in the second graph")

    def step():
        out, lse = E.e3conv_attention(q, k, v, p, p)
        return [t.clone() for t in (out, lse) + E.e3conv_attention_backward(q, k, v, out, lse, g, p, p)]

    want = step()
    a, b = lens[0], lens[0] + lens[1]
    q[a, 0, 1], k[b - 1, 1, 0], v[a + 3, 0, -1], g[b - 1, 2, 3] = float("nan"), float("-inf"), float("inf"), float("nan")
    got = step()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x[:a], y[:a]) and torch.equal(x[b:], y[b:])
