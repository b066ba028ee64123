"""The autograd functions of attention and group norm notice a buffer of theirs that is written between forward
and backward, offsets and masks too (CPU: the library's calls are stood in for, the functions are the real ones)."""

import pytest

from equivariant_gnn_message_amd import e3conv as E


@pytest.fixture
def torch_(monkeypatch):
    import torch
    monkeypatch.setattr(E, "e3conv_attention", lambda q, k, v, *a: (q + v.sum(), torch.zeros(q.shape[:2])))
    monkeypatch.setattr(E, "e3conv_attention_backward", lambda q, k, v, *a: (q, k, v))
    stats = torch.zeros(2, 2)
    monkeypatch.setattr(E, "e3conv_group_norm", lambda x, *a: (x + 0, stats, stats))
    monkeypatch.setattr(E, "e3conv_group_norm_backward", lambda x, p, groups, w, b, *a: (x, w, b))
    return torch


def attend(torch):
    """(result, the buffers it keeps by name)."""
    p, kp = torch.tensor([0, 2, 3], dtype=torch.int32), torch.tensor([0, 1, 3], dtype=torch.int32)
    m = [torch.ones(3, dtype=torch.uint8) for _ in range(2)]
    q, k, v = (torch.ones(3, 2, 4, requires_grad=True) for _ in range(3))
    kept = {"q_ptr": p, "k_ptr": kp, "q_mask": m[0], "k_mask": m[1], "q": q, "k": k, "v": v}
    return E.AttentionFunction.apply(q, k, v, p, kp, 0.5, *m), kept


def norm(torch):
    p, m = torch.tensor([0, 2, 3], dtype=torch.int32), torch.ones(3, dtype=torch.bool)
    x = torch.ones(3, 4, requires_grad=True)
    w, b = (torch.ones(4, requires_grad=True) for _ in range(2))
    return E.GroupNormFunction.apply(x, p, 2, w, b, 1e-5, "silu", m), {"row_ptr": p, "row_mask": m, "x": x, "weight": w}


@pytest.mark.parametrize("make,name", [(attend, n) for n in ("q_ptr", "k_ptr", "q_mask", "k_mask", "q", "k", "v")]
                         + [(norm, n) for n in ("row_ptr", "row_mask", "x", "weight")])
def test_a_written_buffer_is_an_error(torch_, make, name):
    y, kept = make(torch_)
    y.sum().backward()                       # untouched: fine
    y, kept = make(torch_)
    with torch_.no_grad():
        kept[name].zero_()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("make", [attend, norm])
def test_saved_tensor_hooks_see_offsets_and_masks(torch_, make):
    seen = []
    with torch_.autograd.graph.saved_tensors_hooks(lambda t: (seen.append(t.data_ptr()), t)[1], lambda t: t):
        y, kept = make(torch_)
    assert {t.data_ptr() for t in kept.values()} <= set(seen)
    y.sum().backward()


def test_without_masks_and_affine(torch_):
    torch = torch_
    p = torch.tensor([0, 3], dtype=torch.int32)
    q = torch.ones(3, 2, 4, requires_grad=True)
    E.AttentionFunction.apply(q, q, q, p, p).sum().backward()
    x = torch.ones(3, 4, requires_grad=True)
    E.GroupNormFunction.apply(x, p, 2).sum().backward()
    assert q.grad.shape == q.shape and x.grad.shape == x.shape
