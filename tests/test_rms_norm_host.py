"""Refusals of the root-mean-square norm's entry points, without a device (no call gets to a launch), and the
values of its oracle against differences."""

import ctypes

import numpy as np
import pytest

from oracle import rms
from equivariant_gnn_message_amd import e3conv as E

FAKE = 0x1000      # never read: each call fails before any launch


def args_of(**change):
    a = E.RMSNormArgs(dtype=0, channels=32, groups=4, weight_channels=8, eps=1e-5, num_rows=10, x=FAKE, x_row=32,
                      weight=FAKE)
    for name, value in change.items():
        setattr(a, name, value)
    return a


BAD_SIZES = [dict(dtype=2), dict(num_rows=-1), dict(channels=0), dict(channels=65540, groups=10),
             dict(channels=16384, groups=1, weight_channels=1), dict(groups=0), dict(groups=-4), dict(groups=5),
             dict(weight_channels=0), dict(weight_channels=-8), dict(weight_channels=5), dict(weight_channels=64),
             dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(num_rows=1 << 31),
             dict(num_rows=1 << 29)]


def forward(a, y=FAKE, y_row=32, total=None, total_row=0, rstd=FAKE):
    return E.load_library().e3conv_rms_norm(a if a is None else ctypes.byref(a), y, y_row, total, total_row, rstd, None)


def backward(a, rstd=FAKE, gy=FAKE, gy_row=32, gt=None, gt_row=0, gx=FAKE, gx_row=32, gw=FAKE, ws=FAKE, n=1 << 40):
    return E.load_library().e3conv_rms_norm_backward(a if a is None else ctypes.byref(a), rstd, gy, gy_row, gt, gt_row,
                                                     gx, gx_row, gw, ws, n, None)


@pytest.mark.parametrize("change", BAD_SIZES + [dict(x=None), dict(x_row=-1), dict(residual=FAKE, residual_row=-1)],
                         ids=str)
def test_refuses(change):
    a = args_of(**change)
    assert forward(a) == 1 and E.e3conv_last_error_detail()
    assert backward(a) == 1
    if change in BAD_SIZES:
        with pytest.raises(E.E3ConvError) as e:
            E.e3conv_rms_norm_workspace_size(a)
        assert e.value.status == 1


def test_refuses_outputs_and_workspace():
    a = args_of()
    assert forward(None) == 1 and backward(None) == 1
    assert forward(a, y=None) == 1 and forward(a, y_row=-1) == 1 and forward(a, total=FAKE, total_row=-1) == 1
    for name in ("rstd", "gy", "gx"):
        assert backward(a, **{name: None}) == 1
    for name in ("gy_row", "gt_row", "gx_row"):
        assert backward(a, **{name: -1}) == 1
    assert backward(args_of(residual=FAKE, residual_row=32)) == 1
    assert backward(a, ws=None, n=0) == 6 and backward(a, n=8) == 6 and "bytes" in E.e3conv_last_error_detail()
    assert E.load_library().e3conv_rms_norm_workspace_size(ctypes.byref(a), None) == 1


def test_without_rows_is_a_no_op():
    a = args_of(num_rows=0, x=None)
    assert forward(a, y=None, rstd=None) == 0
    assert backward(a, rstd=None, gy=None, gx=None, gw=None, ws=None, n=0) == 0


@pytest.mark.parametrize("rows,channels,groups,period", [(0, 1, 1, 1), (1, 65536, 8, 65536), (1 << 24, 8, 1, 8),
                                                         (1 << 20, 300, 300, 300), (5, 300, 300, 1), (100, 1536, 96, 512)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_workspace_of_any_sizes(rows, channels, groups, period, dtype):
    a = args_of(num_rows=rows, channels=channels, groups=groups, weight_channels=period, dtype=dtype)
    n = E.e3conv_rms_norm_workspace_size(a)
    assert n >= 4 * period and n % 16 == 0


def test_python_refusals():
    import torch
    x = torch.ones((4, 8))
    with pytest.raises(ValueError):
        E.e3conv_rms_norm(x)                       # a host tensor
    with pytest.raises(ValueError):
        E.e3conv_rms_norm(x[0])
    with pytest.raises(TypeError):
        E.e3conv_rms_norm(x.half())


def test_counter_records_stay_valid(tmp_path, monkeypatch):
    """The convolution's counter records are keyed by its own sources."""
    import bench
    csrc = tmp_path / "equivariant_gnn_message_amd" / "csrc"
    csrc.mkdir(parents=True)
    (csrc / "k.hip").write_text("__global__ void k() {}\n")
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    before = bench.kernel_source_hash()
    (csrc / "rms_norm.hip").write_text("__global__ void a() {}\n")
    (csrc / "row_units.h").write_text("int b;\n")
    assert bench.kernel_source_hash() == before


@pytest.mark.parametrize("c,groups,period", [(12, 1, 12), (12, 3, 4), (12, 2, 4), (12, 1, 3), (12, 12, 1)])
@pytest.mark.parametrize("masked", [False, True])
def test_oracle_gradient_is_a_difference(c, groups, period, masked):
    rng = np.random.default_rng(1)
    n, h = 7, 1e-6
    x, res, g, gt, d = rng.standard_normal((5, n, c))
    w, dw = rng.standard_normal((2, period))
    mask = (rng.random(n) < 0.6).astype(np.uint8) if masked else None

    def loss(t, weight):
        v, _ = rms.rms_norm(t, groups, weight, 1e-5, res, mask)
        return (v["y"] * g).sum() + (v["total"] * gt).sum()

    v, _ = rms.rms_norm(x, groups, w, 1e-5, res, mask)
    b, _ = rms.rms_norm_backward(v["total"], groups, w, v["rstd"], g, gt, mask)
    slope = (loss(x + h * d, w + h * dw) - loss(x - h * d, w - h * dw)) / (2 * h)
    np.testing.assert_allclose((b["dx"] * d).sum() + (b["dw"] * dw).sum(), slope, rtol=1e-7, atol=1e-7)


def test_oracle_norm_commutes_with_rotations():
    """An l = 1 block as one group with a weight a channel."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 3, 8))
    turn, _ = np.linalg.qr(rng.standard_normal((3, 3)))
    w = rng.standard_normal(8)
    f = lambda t: rms.rms_norm(t.reshape(5, 24), 1, w)[0]["y"].reshape(5, 3, 8)
    np.testing.assert_allclose(f(np.einsum("ij,njc->nic", turn, x)), np.einsum("ij,njc->nic", turn, f(x)), atol=1e-12)


def test_refuses_one_array_for_both_results():
    """x may take y or the sum, not both."""
    assert forward(args_of(residual=FAKE, residual_row=32), FAKE, 32, FAKE, 32) == 1
    assert "one array" in E.e3conv_last_error_detail()
