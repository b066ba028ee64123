"""Sizes that the attention and group-norm entry points refuse before anything is launched (no device)."""

import ctypes

import pytest

from equivariant_gnn_message_amd import e3conv as E

from .test_graph_ops_host import FAKE, attention_args, norm_args


@pytest.mark.parametrize("change", [dict(num_graphs=1 << 20, channels=4096, groups=4096), dict(num_graphs=1 << 30)],
                         ids=str)
def test_group_norm_pairs_fit_int32(change):
    lib, a = E.load_library(), norm_args(**change)
    ref = ctypes.byref(a)
    assert lib.e3conv_group_norm(ref, FAKE, 4096, None, None, FAKE, 1 << 62, None) == 1
    assert lib.e3conv_group_norm_backward(ref, FAKE, FAKE, FAKE, 4096, FAKE, 4096, None, None, FAKE, 1 << 62, None) == 1
    with pytest.raises(E.E3ConvError):
        E.e3conv_group_norm_workspace_size(a, True)


def test_attention_graphs():
    lib, a = E.load_library(), attention_args(num_graphs=1 << 20)
    assert lib.e3conv_attention(ctypes.byref(a), FAKE, 64, 16, None, FAKE, 1 << 62, None) == 1
