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
