"""Refusals of the attention and group-norm entry points, without a device (no call gets to a launch)."""

import ctypes

import pytest

from equivariant_gnn_message_amd import e3conv as E

FAKE = 0x1000      # never read: each call fails before any launch


def attention_args(**change):
    a = E.AttentionArgs(dtype=0, num_graphs=2, heads_q=4, heads_kv=2, dim_qk=16, dim_v=16, num_q=10, num_k=10,
                        scale=0.25, q_ptr=FAKE, k_ptr=FAKE, q=FAKE, k=FAKE, v=FAKE, q_row=64, q_head=16, k_row=32,
                        k_head=16, v_row=32, v_head=16)
    for name, value in change.items():
        setattr(a, name, value)
    return a


def norm_args(**change):
    a = E.GroupNormArgs(dtype=0, num_graphs=2, channels=32, groups=4, activation=2, eps=1e-5, num_rows=10,
                        row_ptr=FAKE, x=FAKE, x_row=32)
    for name, value in change.items():
        setattr(a, name, value)
    return a


BAD_SIZES = [dict(dtype=2), dict(num_graphs=-1), dict(num_q=-1), dict(num_k=-1), dict(num_graphs=0),
             dict(heads_q=3), dict(heads_q=0), dict(heads_kv=0), dict(dim_qk=0), dict(dim_qk=129), dict(dim_v=0),
             dict(dim_v=129), dict(num_q=1 << 30), dict(num_k=1 << 31), dict(scale=float("nan")),
             dict(scale=float("inf"))]


@pytest.mark.parametrize("change", BAD_SIZES + [dict(q_row=-1), dict(v_head=-16), dict(q=None), dict(k=None),
                                                dict(v=None), dict(q_ptr=None), dict(k_ptr=None)], ids=str)
def test_attention_refuses(change):
    lib = E.load_library()
    a = attention_args(**change)
    assert lib.e3conv_attention(ctypes.byref(a), FAKE, 64, 16, None, FAKE, 1 << 40, None) == 1
    assert E.e3conv_last_error_detail()
    strides = (ctypes.c_int64 * 10)(*[64, 16] * 3 + [32, 16] * 2)
    assert lib.e3conv_attention_backward(ctypes.byref(a), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, strides, FAKE, 1 << 40,
                                         None) == 1
    if change in BAD_SIZES:
        with pytest.raises(E.E3ConvError) as e:
            E.e3conv_attention_workspace_size(a)
        assert e.value.status == 1


def test_attention_refuses_outputs_and_workspace():
    lib = E.load_library()
    a = attention_args(num_q=100000, num_k=100000)
    ref, null = ctypes.byref(a), None
    assert lib.e3conv_attention(null, FAKE, 64, 16, None, None, 0, None) == 1
    assert lib.e3conv_attention(ref, null, 64, 16, None, FAKE, 1 << 40, None) == 1
    assert lib.e3conv_attention(ref, FAKE, -64, 16, None, FAKE, 1 << 40, None) == 1
    good = [64, 16] * 3 + [32, 16] * 2
    back = lambda args, strides, ws=(FAKE, 1 << 40): lib.e3conv_attention_backward(ref, *args, strides, *ws, None)
    every, strides = [FAKE] * 6, (ctypes.c_int64 * 10)(*good)
    for i in range(6):
        assert back([null if j == i else FAKE for j in range(6)], strides) == 1
    assert back(every, null) == 1
    assert back(every, (ctypes.c_int64 * 10)(*good[:9], -1)) == 1
    assert back(every, strides, (null, 0)) == 6 and back(every, strides, (FAKE, 8)) == 6
    assert "bytes" in E.e3conv_last_error_detail()
    assert E.e3conv_attention_workspace_size(a, True) >= 100000 * 4 * 4
    assert lib.e3conv_attention_workspace_size(ref, 0, null) == 1


def test_attention_without_rows_is_a_no_op():
    lib = E.load_library()
    a = attention_args(num_q=0, num_k=0, q=None, k=None, v=None)
    assert lib.e3conv_attention(ctypes.byref(a), None, 0, 0, None, None, 0, None) == 0
    strides = (ctypes.c_int64 * 10)()
    assert lib.e3conv_attention_backward(ctypes.byref(a), *[None] * 6, strides, None, 0, None) == 0


BAD_NORM = [dict(dtype=7), dict(num_graphs=-1), dict(num_rows=-1), dict(num_graphs=0), dict(channels=0),
            dict(channels=4100, groups=1), dict(groups=0), dict(groups=5), dict(activation=4), dict(activation=-1),
            dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(num_rows=1 << 31)]


@pytest.mark.parametrize("change", BAD_NORM + [dict(x_row=-1), dict(x=None), dict(row_ptr=None)], ids=str)
def test_group_norm_refuses(change):
    lib = E.load_library()
    a = norm_args(**change)
    ref = ctypes.byref(a)
    assert lib.e3conv_group_norm(ref, FAKE, 32, None, None, FAKE, 1 << 40, None) == 1
    assert lib.e3conv_group_norm_backward(ref, FAKE, FAKE, FAKE, 32, FAKE, 32, None, None, FAKE, 1 << 40, None) == 1
    if change in BAD_NORM:
        with pytest.raises(E.E3ConvError):
            E.e3conv_group_norm_workspace_size(a, True)


def test_group_norm_refuses_outputs():
    lib = E.load_library()
    a = norm_args()
    ref, big = ctypes.byref(a), (FAKE, 1 << 40, None)
    assert lib.e3conv_group_norm(None, FAKE, 32, None, None, *big) == 1
    assert lib.e3conv_group_norm(ref, None, 32, None, None, *big) == 1
    assert lib.e3conv_group_norm(ref, FAKE, -1, None, None, *big) == 1
    for args in ((None, FAKE, FAKE, 32, FAKE, 32), (FAKE, None, FAKE, 32, FAKE, 32), (FAKE, FAKE, None, 32, FAKE, 32),
                 (FAKE, FAKE, FAKE, 32, None, 32), (FAKE, FAKE, FAKE, -1, FAKE, 32), (FAKE, FAKE, FAKE, 32, FAKE, -1)):
        assert lib.e3conv_group_norm_backward(ref, *args, None, None, *big) == 1
    assert lib.e3conv_group_norm_workspace_size(ref, 0, None) == 1


def test_group_norm_refuses_a_small_workspace():
    lib = E.load_library()
    a = norm_args(num_rows=1 << 20, x_row=32)
    ref = ctypes.byref(a)
    for ws in ((None, 0), (FAKE, 16)):
        assert lib.e3conv_group_norm(ref, FAKE, 32, None, None, *ws, None) == 6
        assert lib.e3conv_group_norm_backward(ref, FAKE, FAKE, FAKE, 32, FAKE, 32, None, None, *ws, None) == 6


def test_host_tensors_are_refused():
    import torch
    t, p = torch.ones((4, 2, 8)), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        E.e3conv_attention(t, t, t, p, p)
    with pytest.raises(ValueError):
        E.e3conv_group_norm(t[:, 0], p, 2)


@pytest.mark.parametrize("num_q,num_k,graphs", [(0, 0, 0), (0, 0, 3), (0, 70000, 3), (70000, 0, 1), (1, 100000, 1),
                                                (100000, 1, 1), (5, 5, 1 << 19)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_attention_workspace_of_any_sizes(num_q, num_k, graphs, dtype):
    a = attention_args(dtype=dtype, num_q=num_q, num_k=num_k, num_graphs=graphs)
    assert E.e3conv_attention_workspace_size(a) >= 0
    assert E.e3conv_attention_workspace_size(a, True) >= 0


@pytest.mark.parametrize("rows,graphs", [(0, 0), (0, 5), (1, 1), (1 << 24, 1), (100, 1 << 19)])
def test_group_norm_workspace_of_any_sizes(rows, graphs):
    a = norm_args(num_rows=rows, num_graphs=graphs)
    assert E.e3conv_group_norm_workspace_size(a) >= 0 and E.e3conv_group_norm_workspace_size(a, True) >= 0


def test_sources_of_these_operators_leave_the_counter_records_valid(tmp_path, monkeypatch):
    """The convolution's counter records are keyed by its own sources."""
    import bench
    csrc = tmp_path / "equivariant_gnn_message_amd" / "csrc"
    csrc.mkdir(parents=True)
    (csrc / "k.hip").write_text("__global__ void k() {}\n")
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    before = bench.kernel_source_hash()
    (csrc / "attention.hip").write_text("__global__ void a() {}\n")
    (csrc / "group_norm.hip").write_text("__global__ void g() {}\n")
    assert bench.kernel_source_hash() == before
