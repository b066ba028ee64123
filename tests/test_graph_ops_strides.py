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
