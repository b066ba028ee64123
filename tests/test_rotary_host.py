"""Refusals of the rotary entry points, without a device (no call gets to a launch), and the values of their oracle
against differences."""

import ctypes

import numpy as np
import pytest

from oracle import rotary
from equivariant_gnn_message_amd import e3conv as E

FAKE = 0x1000      # never read: each call fails before any launch


def args_of(**change):
    a = E.RotaryArgs(dtype=0, layout=0, heads=4, dim=16, pairs=8, axes=3, num_rows=10, x=FAKE, x_row=64, x_head=16,
                     positions=FAKE, position_row=3, waves=FAKE)
    for name, value in change.items():
        setattr(a, name, value)
    return a


BAD_SIZES = [dict(dtype=2), dict(layout=2), dict(layout=-1), dict(num_rows=-1), dict(dim=0), dict(dim=257), dict(dim=15),
             dict(heads=0), dict(heads=65537), dict(pairs=0), dict(pairs=9), dict(axes=0), dict(axes=5),
             dict(num_rows=1 << 31)]


def forward(a, out=FAKE, row=64, head=16):
    return E.load_library().e3conv_rotary(a if a is None else ctypes.byref(a), out, row, head, None)


def backward(a, g=FAKE, gx=FAKE, gp=FAKE, gw=FAKE, strides=(64, 16, 64, 16), ws=FAKE, n=1 << 40):
    return E.load_library().e3conv_rotary_backward(a if a is None else ctypes.byref(a), g, *strides[:2], gx,
                                                   *strides[2:], gp, gw, ws, n, None)


@pytest.mark.parametrize("change", BAD_SIZES + [dict(x=None), dict(positions=None), dict(waves=None), dict(x_row=-1),
                                                dict(x_head=-1), dict(position_row=-1),
                                                dict(x_row=1 << 32), dict(x_head=1 << 32)], ids=str)
def test_refuses(change):
    a = args_of(**change)
    assert forward(a) == 1 and E.e3conv_last_error_detail()
    assert backward(a) == 1
    if change in BAD_SIZES:
        with pytest.raises(E.E3ConvError) as e:
            E.e3conv_rotary_workspace_size(a)
        assert e.value.status == 1


def test_refuses_outputs_and_workspace():
    a = args_of()
    assert forward(None) == 1 and backward(None) == 1
    assert forward(a, out=None) == 1 and forward(a, row=-1) == 1 and forward(a, head=-1) == 1
    assert forward(a, row=1 << 32) == 1 and forward(a, head=1 << 32) == 1
    assert backward(a, g=None) == 1 and backward(a, gx=None) == 1
    for i in range(4):
        assert backward(a, strides=[-1 if i == j else 16 for j in range(4)]) == 1
        assert backward(a, strides=[1 << 32 if i == j else 16 for j in range(4)]) == 1
    assert backward(a, ws=None, n=0) == 6 and backward(a, n=8) == 6 and "bytes" in E.e3conv_last_error_detail()
    assert E.load_library().e3conv_rotary_workspace_size(ctypes.byref(a), None) == 1


def test_without_rows_is_a_no_op():
    a = args_of(num_rows=0, x=None, positions=None)
    assert forward(a, out=None) == 0
    assert backward(a, g=None, gx=None, gp=None, gw=None, ws=None, n=0) == 0


@pytest.mark.parametrize("rows,heads,dim,pairs", [(0, 1, 2, 1), (1, 65536, 256, 128), ((1 << 31) - (1 << 21), 1, 2, 1)])
def test_workspace_of_any_sizes(rows, heads, dim, pairs):
    n = E.e3conv_rotary_workspace_size(args_of(num_rows=rows, heads=heads, dim=dim, pairs=pairs))
    assert n % 16 == 0 and n >= (8 * pairs * 3 if rows else 0)


def test_python_refusals():
    import torch
    x, p, w = torch.ones(4, 2, 8), torch.ones(4, 3), torch.ones(4, 3)
    with pytest.raises(ValueError):
        E.e3conv_rotary(x, p, w)                       # host tensors
    with pytest.raises(ValueError):
        E.e3conv_rotary(x[0], p, w)
    with pytest.raises(TypeError):
        E.e3conv_rotary(x.half(), p, w)


@pytest.mark.parametrize("layout", ["adjacent", "halves"])
def test_oracle_gradient_is_a_difference(layout):
    rng = np.random.default_rng(1)
    n, h = 6, 1e-6
    x, g, d = rng.standard_normal((3, n, 2, 11))
    p, dp = rng.standard_normal((2, n, 3))
    w, dw = rng.standard_normal((2, 4, 3))
    mask = np.array([1, 1, 0, 1, 1, 1])
    loss = lambda t: (rotary.rotary(x + t * d, p + t * dp, w + t * dw, layout, mask)[0] * g).sum()
    v, _ = rotary.rotary_backward(x, p, w, g, layout, mask)
    got = (v["dx"] * d).sum() + (v["dp"] * dp).sum() + (v["dw"] * dw).sum()
    np.testing.assert_allclose(got, (loss(h) - loss(-h)) / (2 * h), rtol=1e-7, atol=1e-7)


def test_oracle_turns_by_the_angle():
    """A quarter turn of each layout, elements beyond the pairs as they are."""
    x = np.arange(1.0, 6.0).reshape(1, 1, 5)
    p, w = np.array([[0.5, 1.0]]), np.array([[np.pi, 0.0], [0.0, np.pi / 2]])
    np.testing.assert_allclose(rotary.rotary(x, p, w)[0][0, 0], [-2, 1, -4, 3, 5], atol=1e-15)
    np.testing.assert_allclose(rotary.rotary(x, p, w, "halves")[0][0, 0], [-3, -4, 1, 2, 5], atol=1e-15)
