"""Arguments that the Python calls of attention and group norm have to refuse with the library's error (host: the
tensors are stand-ins for device ones, and no call gets to a launch)."""

import pytest

from equivariant_gnn_message_amd import e3conv as E


@pytest.fixture
def on_device(monkeypatch):
    """Host tensors pass for tensors on cuda:0."""
    import torch

    class Fake(torch.Tensor):
        def get_device(self):
            return 0

    E.load_library()
    monkeypatch.setattr(E, "_enter", lambda index, stream: (0, None))
    return lambda *shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype).as_subclass(Fake)


def test_head_dimension_of_zero(on_device):
    import torch
    q, p = on_device(4, 2, 0), on_device(2, dtype=torch.int32)
    for call in (lambda: E.e3conv_attention(q, q, q, p, p), lambda: E.e3conv_attention(q, q, q, p, p, 1.0)):
        with pytest.raises(E.E3ConvError) as e:
            call()
        assert e.value.status == 1


@pytest.mark.parametrize("groups", [-1, 0, 3, -8])
def test_group_numbers(on_device, groups):
    import torch
    x, p = on_device(4, 8), on_device(2, dtype=torch.int32)
    stats = on_device(1, 8)
    for call in (lambda: E.e3conv_group_norm(x, p, groups),
                 lambda: E.e3conv_group_norm_backward(x, p, groups, None, None, "none", stats, stats, x)):
        with pytest.raises((E.E3ConvError, ValueError)) as e:
            call()
        assert isinstance(e.value, ValueError) or e.value.status == 1
