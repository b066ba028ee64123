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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("graphs", [0, 2])
def test_backward_of_a_sum_over_no_rows(dtype, graphs):
    """A batch without nodes: the gradient of a sum is an expanded number, without a stride along any axis."""
    import torch
    p = torch.zeros(graphs + 1, dtype=torch.int32, device="cuda")
    leaf = lambda *shape, kind=dtype_of(dtype): torch.ones(shape, dtype=kind, device="cuda", requires_grad=True)
    f32 = torch.float32

    def attend():
        x = [leaf(0, 4, 16), leaf(0, 2, 16), leaf(0, 2, 24)]
        return E.AttentionFunction.apply(*x, p, p), x

    def differ():
        x = [leaf(0, 4, 16), leaf(0, 4, 16), leaf(0, 2, 24), leaf(2, kind=f32)]
        return E.DiffAttentionFunction.apply(*x, p, p), x

    def group_norm():
        x = [leaf(0, 32), leaf(32, kind=f32), leaf(32, kind=f32)]
        return E.GroupNormFunction.apply(x[0], p, 4, *x[1:]), x

    def rms_norm():
        x = [leaf(0, 32), leaf(8, kind=f32)]
        return E.RMSNormFunction.apply(*x, 4), x

    def rms_norm_residual():
        x = [leaf(0, 32), leaf(8, kind=f32), leaf(0, 32)]
        y, total = E.RMSNormFunction.apply(x[0], x[1], 4, 1e-5, x[2])
        return torch.cat([y, total]), x

    def turn():
        x = [leaf(0, 2, 16), leaf(0, 3, kind=f32), leaf(8, 3, kind=f32)]
        return E.RotaryFunction.apply(*x), x

    for call in (attend, differ, group_norm, rms_norm, rms_norm_residual, turn):
        y, x = call()
        y.sum().backward()
        torch.cuda.synchronize()
        assert all(t.grad.shape == t.shape and bool((t.grad == 0).all()) for t in x), call.__name__
