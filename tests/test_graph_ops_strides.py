"""Strides that the Python calls beside the convolution take and give (host tensors stand in for device ones)."""

import itertools

import pytest

from equivariant_gnn_message_amd import e3conv as E

from .test_graph_ops_arguments import on_device  # noqa: F401  (fixture)


def test_operands_without_elements_may_have_any_strides(on_device):
    """The gradient of a sum over no rows is an expanded number, and contiguous as it is."""
    import torch
    g = on_device(1)[0].expand(0, 2, 16)
    assert g.contiguous().stride(-1) == 0
    assert E._rows_of(g, "grad_out", torch.float32, 0, (0, 2, 16)) == (0, 0, 0)
    with pytest.raises(ValueError, match="unit stride"):
        E._rows_of(on_device(1)[0].expand(3, 2, 16), "grad_out", torch.float32, 0, (3, 2, 16))


def test_gradients_of_overlapping_operands_are_dense():
    """Sliding windows, repeated heads: a gradient allocated for one has unit stride along its last axis and no element
    twice (an empty_like of such windows has neither)."""
    import torch
    base = torch.zeros(100)
    for shape in itertools.product((0, 1, 2, 3), (1, 2, 3), (1, 2, 4)):
        for strides in itertools.product((0, 1, 2, 4, 8, 16), (0, 1, 2, 4, 8), (1, 3)):
            if strides[2] != 1 and shape[2] > 1:
                continue
            g = E._gradient_like(base.as_strided(shape, strides))
            at = [sum(a * b for a, b in zip(i, g.stride())) for i in itertools.product(*map(range, shape))]
            assert g.shape == shape and (shape[2] <= 1 or g.numel() == 0 or g.stride(2) == 1), (shape, strides)
            assert len(set(at)) == len(at) and max(at, default=-1) < max(g.untyped_storage().nbytes() // 4, 1)
    packed = torch.zeros(5, 3, 4)
    assert E._gradient_like(packed).stride() == packed.stride()
    assert E._gradient_like(packed.transpose(0, 1)).stride() == packed.transpose(0, 1).stride()
