"""Batches without graphs or rows through the operators beside the convolution, their reverse passes and autograd."""

import pytest

from equivariant_gnn_message_amd import e3conv as E

from .test_gpu_attention import dtype_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,dv", [(16, 32), (64, 128)])
def test_differential_attention_without_graphs(dtype, d, dv):
    """Offsets [0]: no graph, no row; the gradient of lambda is zero, and written."""
    import torch
    p = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, v = (torch.zeros(0, h, n, dtype=dtype_of(dtype), device="cuda") for h, n in ((4, d), (2, dv)))
    lam = torch.ones(2, device="cuda")
    torch.full((1024,), 7.0, device="cuda")              # freed: what lambda's gradient may be allocated over
    out, second, lse = E.e3conv_diff_attention(q, q, v, lam, p, p)
    grads = E.e3conv_diff_attention_backward(q, q, v, lam, out, second, lse, v, p, p)
    torch.cuda.synchronize()
    assert [t.shape for t in grads] == [t.shape for t in (q, q, v, lam)] and bool((grads[3] == 0).all())
