"""The autograd functions of the root-mean-square norm, the rotary positions and differential attention notice a buffer
of theirs that is written between forward and backward, and the Python calls refuse bad arguments with the library's
error (CPU: the library's calls are stood in for, the functions are the real ones)."""

import pytest

from equivariant_gnn_message_amd import e3conv as E

from .test_graph_ops_arguments import on_device  # noqa: F401  (fixture)


@pytest.fixture
def torch_(monkeypatch):
    import torch
    some = torch.zeros(3, 2)
    monkeypatch.setattr(E, "e3conv_diff_attention", lambda q, k, v, lam, *a: (v + q.sum(), v + 0, some))
    monkeypatch.setattr(E, "e3conv_diff_attention_backward", lambda q, k, v, lam, *a: (q, k, v, lam))
    monkeypatch.setattr(E, "e3conv_rms_norm", lambda x, w, groups, eps, r, m: (x + 0, None if r is None else x + r, some))
    monkeypatch.setattr(E, "e3conv_rms_norm_backward", lambda x, w, *a: (x, w))
    monkeypatch.setattr(E, "e3conv_rotary", lambda x, *a: x + 0)
    monkeypatch.setattr(E, "e3conv_rotary_backward", lambda x, p, w, *a, **k: (x, p, w))
    return torch


def attend(torch):
    """(result, the buffers it keeps by name)."""
    p, kp = torch.tensor([0, 2, 3], dtype=torch.int32), torch.tensor([0, 1, 3], dtype=torch.int32)
    m = [torch.ones(3, dtype=torch.uint8) for _ in range(2)]
    q, k, v = (torch.ones(3, h, 4, requires_grad=True) for h in (4, 4, 2))
    lam = torch.ones(2, requires_grad=True)
    kept = {"q_ptr": p, "k_ptr": kp, "q_mask": m[0], "k_mask": m[1], "q": q, "k": k, "v": v, "lam": lam}
    return E.DiffAttentionFunction.apply(q, k, v, lam, p, kp, 0.5, *m), kept


def norm(torch):
    m, x, w = torch.ones(3, dtype=torch.bool), torch.ones(3, 4, requires_grad=True), torch.ones(4, requires_grad=True)
    return E.RMSNormFunction.apply(x, w, 2, 1e-5, None, m), {"row_mask": m, "x": x, "weight": w}


def turn(torch):
    m, x = torch.ones(3, dtype=torch.bool), torch.ones(3, 2, 4, requires_grad=True)
    p, w = torch.ones(3, 3, requires_grad=True), torch.ones(2, 3, requires_grad=True)
    return E.RotaryFunction.apply(x, p, w, "halves", m), {"row_mask": m, "x": x, "positions": p, "waves": w}


@pytest.mark.parametrize("make,name", [(attend, n) for n in ("q_ptr", "k_ptr", "q_mask", "k_mask", "q", "k", "v", "lam")]
                         + [(norm, n) for n in ("row_mask", "x", "weight")]
                         + [(turn, n) for n in ("row_mask", "x", "positions", "waves")])
def test_a_written_buffer_is_an_error(torch_, make, name):
    y, kept = make(torch_)
    y.sum().backward()                       # untouched: fine
    y, kept = make(torch_)
    with torch_.no_grad():
        kept[name].zero_()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_total_of_the_norm_is_kept(torch_):
    """With a residual the sum is what the reverse pass reads: writing it is noticed, writing x is not an error."""
    for index, ok in ((0, True), (1, False)):
        x, w, r = (torch_.ones(s, requires_grad=True) for s in ((3, 4), (4,), (3, 4)))
        y, total = E.RMSNormFunction.apply(x, w, 2, 1e-5, r)
        with torch_.no_grad():
            (x, total)[index].zero_()
        if ok:
            y.sum().backward()
        else:
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                y.sum().backward()


def test_without_masks_and_weights(torch_):
    torch = torch_
    x = torch.ones(3, 4, requires_grad=True)
    E.RMSNormFunction.apply(x).sum().backward()
    assert x.grad.shape == x.shape


def test_empty_axes_are_refused(on_device):  # noqa: F811
    import torch
    p, lam = on_device(2, dtype=torch.int32), on_device(2)
    for call in (lambda: E.e3conv_diff_attention(on_device(4, 4, 0), on_device(4, 4, 0), on_device(4, 2, 8), lam, p, p),
                 lambda: E.e3conv_diff_attention(on_device(4, 4, 8), on_device(4, 4, 8), on_device(4, 2, 0), lam, p, p),
                 lambda: E.e3conv_diff_attention(on_device(4, 4, 65), on_device(4, 4, 65), on_device(4, 2, 8), lam, p, p),
                 lambda: E.e3conv_rms_norm(on_device(4, 0)), lambda: E.e3conv_rms_norm(on_device(4, 8), groups=3),
                 lambda: E.e3conv_rms_norm(on_device(4, 8), on_device(3)),
                 lambda: E.e3conv_rotary(on_device(4, 2, 0), on_device(4, 3), on_device(1, 3)),
                 lambda: E.e3conv_rotary(on_device(4, 2, 8), on_device(4, 3), on_device(0, 3)),
                 lambda: E.e3conv_rotary(on_device(4, 2, 8), on_device(4, 5), on_device(2, 5)),
                 lambda: E.e3conv_rotary(on_device(4, 2, 8), on_device(4, 3), on_device(5, 3))):
        with pytest.raises((E.E3ConvError, ValueError)) as e:
            call()
        assert isinstance(e.value, ValueError) or e.value.status == 1
