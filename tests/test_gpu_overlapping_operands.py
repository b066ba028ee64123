"""Sliding windows as operands of attention: rows and heads that overlap in memory, whose gradients do not."""

import pytest

from equivariant_gnn_message_amd import e3conv as E

from .test_gpu_attention import dev, dtype_of, ptr

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("steps", [(1, 40), (3, 1), (0, 1), (1, 0)])
def test_gradients_of_windows(dtype, steps):
    """The bits of the call with copied operands."""
    import torch
    n, d, dv = 33, 16, 24
    gen = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(600, generator=gen).to(dtype_of(dtype)).cuda().as_strided((n, h, w), (*steps, 1))
               for h, w in ((4, d), (4, d), (2, dv)))
    g = torch.randn((n, 4, dv), generator=gen).to(dtype_of(dtype)).cuda()
    lam, p = torch.tensor([0.3, 0.6], device="cuda"), dev(ptr([n - 3, 3]))
    dense = [t.contiguous() for t in (q, k, v)]
    out = E.e3conv_diff_attention(q, k, v, lam, p, p)
    assert all(torch.equal(a, b) for a, b in zip(out, E.e3conv_diff_attention(*dense, lam, p, p)))
    back = E.e3conv_diff_attention_backward
    got, want = (back(*x, lam, *out, g[:, :2], p, p) for x in ((q, k, v), dense))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    k, dense[1] = k[:, :2], dense[1][:, :2]
    out = E.e3conv_attention(q, k, v, p, p)
    got, want = (E.e3conv_attention_backward(*x, *out, g, p, p) for x in ((q, k, v), dense))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
