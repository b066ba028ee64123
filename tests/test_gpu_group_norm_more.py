"""Group norm where its sums and its dispatch can go wrong: outlying rows, rows wider than one work-group, results
larger than the L2s, and more groups than one launch has work-groups.  Bounds: oracle.norm.group_norm."""

import numpy as np
import pytest

from oracle import norm
from equivariant_gnn_message_amd import e3conv as E

from ._gpu import say
from .test_gpu_attention import U, dev, dtype_of, host, ptr

pytestmark = pytest.mark.gpu


def inputs(dtype, lens, channels, seed=0):
    """x, grad_y (device), weight, bias (numpy)."""
    import torch
    gen = torch.Generator().manual_seed(seed + channels)
    n = int(sum(lens))
    x, g = (torch.randn((n, channels), generator=gen).to(dtype_of(dtype)).cuda() for _ in range(2))
    w, b = 1 + 0.3 * torch.randn(channels, generator=gen), 0.3 * torch.randn(channels, generator=gen)
    return x, g, w.numpy(), b.numpy()


def compare(dtype, lens, groups, x, g, w, b, act="silu", mask=None, eps=1e-5, out=None, grad_x=None):
    import torch
    u, r = U[dtype]
    p, m = dev(ptr(lens)), None if mask is None else dev(mask)
    clean = lambda t: host(t) if mask is None else np.where(np.asarray(mask, bool)[:, None], host(t), 0.0)
    val, tol = norm.group_norm(clean(x), ptr(lens), groups, w, b, float(np.float32(eps)), act, mask, clean(g), u, r)
    say(f"[group norm] {dtype} rows {x.shape[0]} in {len(lens)} graphs, {x.shape[1]} channels, {groups} groups, {act}")
    keep = x.clone() if out is x else x
    y, mean, rstd = E.e3conv_group_norm(x, p, groups, dev(w), dev(b), eps, act, m, out=out)
    gx, gw, gb = E.e3conv_group_norm_backward(keep, p, groups, dev(w), dev(b), act, mean, rstd, g, m, grad_x=grad_x)
    torch.cuda.synchronize()
    for name, t in {"mean": mean, "rstd": rstd, "y": y, "dx": gx, "dw": gw, "dc": gb}.items():
        off = np.abs(host(t) - val[name])
        worst = float(np.max(off - tol[name], initial=-1.0))
        say(f"  {name}: max err {float(np.max(off, initial=0.0)):.3e}, over its bound by {worst:.3e}")
        assert bool(np.all(np.isfinite(off))) and worst <= 1e-30, (name, worst)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("big", [100.0, 10000.0])
@pytest.mark.parametrize("lens,channels", [([30000] + [5] * 15, 8), ([20000], 64), ([4000, 3], 64)], ids=str)
@pytest.mark.parametrize("at", [0, 1, 2500])
def test_one_outlying_row(dtype, big, lens, channels, at):
    """A master node far from all others, first in its graph or not; graphs of one chunk and of many."""
    x, g, w, b = inputs(dtype, lens, channels)
    x[at] = big
    compare(dtype, lens, 2, x, g, w, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("big", [100.0, 10000.0])
def test_outlying_row_alone_in_its_chunk(dtype, big):
    """A graph of 16 chunks of 1024 rows; of the first one the mask leaves the master node alone."""
    lens = [16000] * 64
    x, g, w, b = inputs(dtype, lens, 8)
    mask = np.ones(sum(lens), dtype=np.uint8)
    for graph in (0, 7):
        x[16000 * graph] = big
        mask[16000 * graph + 1:16000 * graph + 1024] = 0
    compare(dtype, lens, 2, x, g, w, b, "none", mask)


def single_rows(graphs, channels, groups):
    """Graphs of one row, one in eight masked: with a group's value its own mean, y = bias, dx = 0 but for the
    rounding of dz w, grad_bias the sum of dz, grad_weight = 0."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(graphs)
    x, g = (torch.randn((graphs, channels), generator=gen, device="cuda") for _ in range(2))
    w, b = (torch.rand(channels, generator=gen, device="cuda") + 0.5 for _ in range(2))
    p = torch.arange(graphs + 1, dtype=torch.int32, device="cuda")
    mask = torch.arange(graphs, device="cuda") % 8 != 3
    say(f"[group norm] {graphs} graphs of one row, {channels} channels, {groups} groups")
    return x, g, w, b, p, mask


def test_more_groups_than_one_axis_of_a_launch():
    """5000 graphs x 4096 groups: 20 million (graph, group) pairs of 256 threads are more than 2^32 threads."""
    import torch
    x, g, w, b, p, mask = single_rows(5000, 4096, 4096)
    y, mean, rstd = E.e3conv_group_norm(x, p, 4096, w, b, 1e-2, "none", mask)
    gx, gw, gb = E.e3conv_group_norm_backward(x, p, 4096, w, b, "none", mean, rstd, g, mask)
    torch.cuda.synchronize()
    seen, u = mask[:, None].float(), 2.0 ** -24
    assert torch.equal(mean, x * seen) and bool(((rstd - 10).abs() <= 40 * u).all())
    assert torch.equal(y, b.expand_as(y) * seen)
    assert bool((gx.abs() <= 2 * u * (g * w).abs() * 10 * seen).all()) and not gw.any()
    want, size = (g.double() * seen).sum(0), (g.double().abs() * seen).sum(0)
    assert bool(((gb - want).abs() <= 4 * 5000 ** 0.5 * u * size).all())


def test_more_graphs_than_one_axis_of_a_launch():
    """17 million graphs, a work-group of 256 threads each."""
    import torch
    graphs = 17 << 20
    x, g, w, b, p, mask = single_rows(graphs, 4, 4)
    y, mean, rstd = E.e3conv_group_norm(x, p, 4, w, b, 1e-2, "none", mask)
    gx, gw, gb = E.e3conv_group_norm_backward(x, p, 4, w, b, "none", mean, rstd, g, mask)
    torch.cuda.synchronize()
    seen, u = mask[:, None].float(), 2.0 ** -24
    assert torch.equal(mean, x * seen) and bool(((rstd - 10).abs() <= 40 * u).all())
    assert torch.equal(y, b.expand_as(y) * seen)
    assert bool((gx.abs() <= 2 * u * (g * w).abs() * 10 * seen).all()) and not gw.any()
    want, size = (g.double() * seen).sum(0), (g.double().abs() * seen).sum(0)
    assert bool(((gb - want).abs() <= 4 * graphs ** 0.5 * u * size).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("channels,groups", [(4096, 32), (2056, 8), (2056, 2056), (1028, 4), (300, 300), (300, 12),
                                             (1001, 7), (4095, 9), (257, 257)])
@pytest.mark.parametrize("masked", [False, True])
def test_rows_wider_than_a_work_group(dtype, channels, groups, masked):
    """More than 256 runs of channels: several work-groups along a row, the last one narrower, of whole 16-byte
    runs (fp32 by 4, bf16 by 8) and element by element; with empty graphs and graphs of one chunk and of many."""
    lens = [3, 0, 200, 1, 0]
    mask = None
    if masked:
        mask = (np.random.default_rng(channels).random(sum(lens)) < 0.7).astype(np.uint8)
        mask[-1] = 0
    x, g, w, b = inputs(dtype, lens, channels)
    if masked:
        hole = dev(mask == 0)
        x[hole], g[hole] = float("nan"), float("inf")
    compare(dtype, lens, groups, x, g, w, b, "silu", mask)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("dtype,rows", [("f32", 150000), ("bf16", 300000)])
def test_results_larger_than_the_l2s(dtype, rows, act):
    """Results of more than 32 MiB are stored past the caches, by kernels of their own: out of place, in place, and
    over a mask."""
    lens = [rows - 5000, 0, 4999, 1]
    x, g, w, b = inputs(dtype, lens, 64)
    if act == "relu":      # keep z away from the corner: its derivative is a step there
        z = norm.group_norm(host(x), ptr(lens), 8, w, b, float(np.float32(1e-5)), "none")[0]["y"]
        g[dev(np.abs(z) < 1e-3)] = 0
    compare(dtype, lens, 8, x, g, w, b, act)
    if act == "silu":
        y, gx = x.clone(), g.clone()
        compare(dtype, lens, 8, y, gx, w, b, act, out=y, grad_x=gx)
        mask = (np.arange(rows) % 5 != 2).astype(np.uint8)
        compare(dtype, lens, 8, x, g, w, b, act, mask)
