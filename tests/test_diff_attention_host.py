"""Refusals of the differential attention's entry points, without a device (no call gets to a launch), and the values of
its oracle: against the plain attention's, and against differences."""

import ctypes

import numpy as np
import pytest

from oracle import attention, diff_attention
from equivariant_gnn_message_amd import e3conv as E

from .test_graph_ops_host import FAKE, attention_args


def forward(a, lam=FAKE, out=FAKE, strides=(64, 16, 64, 16), second=FAKE, ws=FAKE, n=1 << 40):
    return E.load_library().e3conv_diff_attention(a if a is None else ctypes.byref(a), lam, out, *strides[:2], second,
                                                  *strides[2:], None, ws, n, None)


def backward(a, given=(FAKE,) * 9, strides=(64, 16) * 6, ws=FAKE, n=1 << 40):
    """given: lambda, out, second, lse, grad_out, grad_q, grad_k, grad_v, grad_lambda."""
    s = None if strides is None else (ctypes.c_int64 * 12)(*strides)
    return E.load_library().e3conv_diff_attention_backward(a if a is None else ctypes.byref(a), *given, s, ws, n, None)


BAD_SIZES = [dict(dtype=2), dict(num_graphs=-1), dict(num_q=-1), dict(num_k=-1), dict(num_graphs=0),
             dict(num_graphs=1 << 20), dict(heads_q=3), dict(heads_q=0), dict(heads_kv=0), dict(dim_qk=0),
             dict(dim_qk=65), dict(dim_v=0), dict(dim_v=129), dict(num_q=1 << 28), dict(num_k=1 << 30),
             dict(scale=float("nan")), dict(scale=float("inf"))]


@pytest.mark.parametrize("change", BAD_SIZES + [dict(q_row=-1), dict(v_head=-16), dict(q=None), dict(k=None),
                                                dict(v=None), dict(q_ptr=None), dict(k_ptr=None)], ids=str)
def test_refuses(change):
    a = attention_args(**change)
    assert forward(a) == 1 and E.e3conv_last_error_detail()
    assert backward(a) == 1
    if change in BAD_SIZES:
        with pytest.raises(E.E3ConvError) as e:
            E.e3conv_diff_attention_workspace_size(a)
        assert e.value.status == 1


def test_refuses_outputs_and_workspace():
    a = attention_args(num_q=100000, num_k=100000)
    assert forward(None) == 1 and backward(None) == 1
    assert forward(a, lam=None) == 1 and forward(a, out=None) == 1
    for i in range(4):
        assert forward(a, strides=[-1 if i == j else 16 for j in range(4)]) == 1
    for i in range(8):
        assert backward(a, [None if i == j else FAKE for j in range(9)]) == 1
    assert backward(a, strides=None) == 1
    for i in range(12):
        assert backward(a, strides=[-1 if i == j else 16 for j in range(12)]) == 1
    assert backward(a, ws=None, n=0) == 6 and backward(a, n=8) == 6
    assert "bytes" in E.e3conv_last_error_detail()
    assert E.load_library().e3conv_diff_attention_workspace_size(ctypes.byref(a), 0, None) == 1


def test_a_split_forward_needs_its_workspace():
    a = attention_args(num_graphs=1, num_q=1, num_k=100000)
    assert E.e3conv_diff_attention_workspace_size(a) > 0
    assert forward(a, ws=None, n=0) == 6 and forward(a, n=16) == 6


def test_without_rows_is_a_no_op():
    a = attention_args(num_q=0, num_k=0, q=None, k=None, v=None)
    assert forward(a, lam=None, out=None, second=None, ws=None, n=0) == 0
    assert backward(a, [None] * 9, ws=None, n=0) == 0


@pytest.mark.parametrize("num_q,num_k,graphs", [(0, 0, 0), (0, 0, 3), (0, 70000, 3), (70000, 0, 1), (1, 100000, 1),
                                                (100000, 1, 1), (5, 5, 1 << 19)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_workspace_of_any_sizes(num_q, num_k, graphs, dtype):
    a = attention_args(dtype=dtype, num_q=num_q, num_k=num_k, num_graphs=graphs)
    for backward_too in (False, True):
        assert E.e3conv_diff_attention_workspace_size(a, backward_too) % 16 == 0


def test_python_refusals():
    import torch
    q, v, p, lam = torch.ones(4, 4, 8), torch.ones(4, 2, 16), torch.tensor([0, 4], dtype=torch.int32), torch.ones(2)
    with pytest.raises(ValueError):
        E.e3conv_diff_attention(q, q, v, lam, p, p)              # host tensors
    with pytest.raises(ValueError):
        E.e3conv_diff_attention(q[:, :3], q, v, lam, p, p)       # an odd number of maps
    with pytest.raises(TypeError):
        E.e3conv_diff_attention(q.half(), q, v, lam, p, p)


def inputs(seed=1, hq=4, hk=2, d=5, dv=7):
    rng = np.random.default_rng(seed)
    q_ptr, k_ptr = np.array([0, 3, 3, 9]), np.array([0, 6, 8, 13])
    q, k = rng.standard_normal((9, 2 * hq, d)), rng.standard_normal((13, 2 * hk, d))
    v, g = rng.standard_normal((13, hk, dv)), rng.standard_normal((9, hq, dv))
    q_mask, k_mask = (rng.random(9) < 0.8).astype(int), (rng.random(13) < 0.7).astype(int)
    return [q, k, v, rng.standard_normal(hq)], g, (q_ptr, k_ptr, 0.4, q_mask, k_mask)


def test_oracle_is_the_difference_of_two_attentions():
    (q, k, v, lam), g, rest = inputs()
    got = diff_attention.diff_attention(q, k, v, lam, *rest, grad=g)
    first = attention.attention(q[:, 0::2], k[:, 0::2], v, *rest, grad=g)
    second = attention.attention(q[:, 1::2], k[:, 1::2], v, *rest, grad=-lam[:, None] * g)
    np.testing.assert_allclose(got["out"], first["out"] - lam[:, None] * second["out"], atol=1e-13)
    np.testing.assert_allclose(got["second"], second["out"], atol=1e-13)
    for m, part in ((0, first), (1, second)):
        np.testing.assert_allclose(got["dq"][:, m::2], part["dq"], atol=1e-13)
        np.testing.assert_allclose(got["dk"][:, m::2], part["dk"], atol=1e-13)
        np.testing.assert_array_equal(np.isneginf(got["lse"][..., m]), np.isneginf(part["lse"]))
    np.testing.assert_allclose(got["dv"], first["dv"] + second["dv"], atol=1e-13)
    np.testing.assert_allclose(got["dlam"], -(g * second["out"]).sum((0, 2)), atol=1e-13)


def test_oracle_gradient_is_a_difference():
    x, g, rest = inputs(2)
    along, _, _ = inputs(3)
    h = 1e-6
    loss = lambda t: (diff_attention.diff_attention(*(a + t * b for a, b in zip(x, along)), *rest)["out"] * g).sum()
    v = diff_attention.diff_attention(*x, *rest, grad=g)
    got = sum((v[n] * b).sum() for n, b in zip(("dq", "dk", "dv", "dlam"), along))
    np.testing.assert_allclose(got, (loss(h) - loss(-h)) / (2 * h), rtol=1e-7, atol=1e-7)
