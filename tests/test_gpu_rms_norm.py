"""The root-mean-square norm with a residual, and its reverse pass, against oracle.rms.

Tolerances are the oracle's elementwise bounds with u = 2^-24 and, for bf16 results, one rounding of 2^-8.
"""

import numpy as np
import pytest

from oracle import rms
from equivariant_gnn_message_amd import e3conv as E

from ._gpu import say
from .test_gpu_attention import U, dev, dtype_of, host

pytestmark = pytest.mark.gpu


def draw(seed, dtype, n, c, scale=1.0):
    import torch
    gen = torch.Generator().manual_seed(seed)
    return (scale * torch.randn((n, c), generator=gen)).to(dtype_of(dtype)).cuda()


def weight_of(period, seed=9):
    import torch
    return (1 + 0.3 * torch.randn(period, generator=torch.Generator().manual_seed(seed))).cuda()


def within(got, want, tol, label):
    for name in got:
        off = np.abs(host(got[name]).reshape(want[name].shape) - want[name])
        assert np.all(np.isfinite(off)), (label, name)
        worst = float(np.max(off - tol[name], initial=-1.0))
        say(f"  {name}: max err {float(np.max(off, initial=0.0)):.3e}, over its bound by {worst:.3e}")
        assert worst <= 1e-30, (label, name, worst)


def check(dtype, x, groups=1, weight=None, eps=1e-5, residual=None, mask=None, g=None, gt=None, label=""):
    """Forward and reverse pass of one call against the oracle; the library's results."""
    import torch
    say(f"[rms] {dtype} {tuple(x.shape)} groups {groups} weight {None if weight is None else weight.numel()} {label}")
    u, r = U[dtype]
    m = None if mask is None else dev(mask)
    y, total, rstd = E.e3conv_rms_norm(x, weight, groups, eps, residual, m)
    torch.cuda.synchronize()
    clean = lambda t: None if t is None else host(t) if mask is None else np.where(mask[:, None] != 0, host(t), 0.0)
    w = None if weight is None else host(weight)
    want, tol = rms.rms_norm(clean(x), groups, w, float(np.float32(eps)), clean(residual), mask, u, r)
    got = {"y": y, "rstd": rstd}
    if residual is not None:
        got["total"] = total
    else:
        assert total is None
    within(got, want, tol, label)
    s = x if total is None else total
    if g is None:
        g = draw(77, dtype, *x.shape)
    gx, gw = E.e3conv_rms_norm_backward(s, weight, groups, rstd, g, gt, m)
    torch.cuda.synchronize()
    want, tol = rms.rms_norm_backward(clean(s), groups, w, host(rstd), clean(g), clean(gt), mask, u, r)
    got = {"dx": gx}
    if weight is not None:
        got["dw"] = gw
    else:
        assert gw is None
    within(got, want, tol, label)
    return y, total, rstd, gx, gw


# channels, groups, weight values: rows, heads that share a weight or have their own, an l-block's components,
# periods that neither divide a group nor are divided by one; sizes around a run, a wave and a work-group
SHAPES = [(1, 1, 1), (2, 1, 2), (7, 1, 7), (8, 1, 8), (24, 3, 8), (24, 1, 8), (24, 3, 24), (33, 1, 11), (64, 4, 16),
          (64, 4, 64), (72, 6, 24), (12, 2, 4), (40, 5, 16 // 2), (504, 1, 72), (512, 4, 128), (512, 4, 512),
          (520, 1, 520), (1024, 1, 1024), (2048, 1, 2048), (2056, 1, 2056), (4100, 1, 4100), (8192, 1, 8192),
          (8191, 1, 8191), (16384, 4, 4096), (1600, 100, 1600), (1536, 96, 512), (300, 300, 300), (300, 300, 1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("c,groups,period", SHAPES)
def test_shapes(dtype, c, groups, period):
    for n, residual in ((1, False), (37, True), (5, False)):
        res = draw(2, dtype, n, c) if residual else None
        check(dtype, draw(1, dtype, n, c), groups, weight_of(period), residual=res,
              gt=draw(3, dtype, n, c) if residual else None)
    check(dtype, draw(4, dtype, 3, c), groups)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,c,groups,period", [(3, 8193, 1, 8193), (19, 10240, 1, 2048), (1500, 10240, 1, 2048), (700, 14336, 1, 2048),
                                               (5, 16383, 1, 16383), (1, 16376, 1, 16376), (31, 20480, 2, 10240),
                                               (9, 36864, 3, 36864), (7, 65532, 4, 16383), (4, 27000, 3, 5)])
def test_wide_groups(dtype, n, c, groups, period):
    """More channels in a group than a work-group of 256 threads holds, up to the limit."""
    check(dtype, draw(1, dtype, n, c), groups, weight_of(period), residual=draw(2, dtype, n, c), gt=draw(3, dtype, n, c))
    mask = (np.random.default_rng(n).random(n) < 0.6).astype(np.uint8)
    check(dtype, draw(4, dtype, n, c), groups, mask=mask)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,c,groups,period", [(70001, 16, 1, 16), (20000, 128, 4, 32), (9001, 24, 3, 24),
                                               (3000, 1600, 100, 1600), (5000, 2304, 1, 768), (100000, 3, 1, 3)])
def test_many_rows(dtype, n, c, groups, period):
    check(dtype, draw(5, dtype, n, c), groups, weight_of(period), residual=draw(6, dtype, n, c), gt=draw(7, dtype, n, c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("c,groups", [(64, 4), (33, 1), (4096, 1)])
def test_masked_rows_hold_anything(dtype, c, groups):
    import torch
    n = 75
    mask = (np.random.default_rng(5).random(n) < 0.7).astype(np.uint8)
    hole = torch.from_numpy(mask == 0).cuda()
    x, res, g, gt = (draw(s, dtype, n, c) for s in (1, 2, 3, 4))
    for t, bad in ((x, float("nan")), (res, float("inf")), (g, float("nan")), (gt, float("-inf"))):
        t[hole] = bad
    y, total, rstd, gx, _ = check(dtype, x, groups, weight_of(c // groups), residual=res, mask=mask, g=g, gt=gt)
    assert all(bool((t[hole] == 0).all()) for t in (y, total, gx))
    assert bool((rstd[hole] == rstd[hole][0, 0]).all()) and abs(float(rstd[hole][0, 0]) * 1e-5 ** 0.5 - 1) < 1e-6
    again = E.e3conv_rms_norm(x, weight_of(c // groups), groups, residual=res, row_mask=~hole)
    assert all(torch.equal(a, b) for a, b in zip(again, (y, total, rstd)))
    none = np.zeros(n, np.uint8)
    y, _, _, gx, gw = check(dtype, x, groups, weight_of(c // groups), mask=none, g=g)
    assert bool((y == 0).all() & (gx == 0).all()) and bool((gw == 0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_values(dtype):
    """Zero rows, tiny and large ones, an outlying channel."""
    x = draw(1, dtype, 9, 200)
    x[0] = 0
    x[1] *= 1e-12
    x[2] *= 1e15
    x[3, 7] = 1e6
    check(dtype, x, 1, weight_of(200), label="values")
    check(dtype, x, 5, weight_of(40), eps=1e-12, label="small eps")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_places(dtype):
    """Rows of wider tensors, unaligned rows, results in place: bit-equal to the dense call."""
    import torch
    n, c = 50, 24
    x, res, g, gt = (draw(s, dtype, n, c) for s in (1, 2, 3, 4))
    w = weight_of(8)
    want = E.e3conv_rms_norm(x, w, 1, residual=res)
    back = E.e3conv_rms_norm_backward(want[1], w, 1, want[2], g, gt)

    def wide(t, spare):
        return torch.cat([t, torch.full((n, spare), 7.0, dtype=t.dtype, device="cuda")], 1)[:, :c]

    block = torch.zeros((n, 4, 8), dtype=x.dtype, device="cuda")
    block[:, 1:] = x.view(n, 3, 8)
    for spare in (8, 1):
        say(f"[rms] {dtype} rows of {c + spare}")
        got = E.e3conv_rms_norm(wide(x, spare), w, 1, residual=wide(res, spare), out=wide(x, spare), total=wide(x, spare))
        gotb = E.e3conv_rms_norm_backward(wide(want[1], spare), w, 1, want[2], wide(g, spare), wide(gt, spare),
                                          grad_x=wide(x, spare))
        tol = dict(rtol=2.0 ** -20, atol=1e-6) if dtype == "f32" else dict(rtol=2.0 ** -7, atol=1e-6)
        for a, b in zip(got + gotb, want + back):       # another form adds in another order
            torch.testing.assert_close(a, b, **tol)
        assert all(bool((t._base[:, c:] == 7).all()) for t in (got[0], got[1], gotb[0]))
    y, _, _ = E.e3conv_rms_norm(block[:, 1:].flatten(1), w, 1)
    assert torch.equal(y, E.e3conv_rms_norm(x, w, 1)[0])
    assert block[:, 1:].flatten(1).data_ptr() == block[:, 1:].data_ptr()          # the block where it lies
    a, b = x.clone(), res.clone()
    got = E.e3conv_rms_norm(a, w, 1, residual=b, out=a, total=b)
    assert got[0] is a and got[1] is b and all(torch.equal(s, t) for s, t in zip(got, want))
    a, b = x.clone(), res.clone()
    got = E.e3conv_rms_norm(a, w, 1, residual=b, out=b, total=a)
    assert all(torch.equal(s, t) for s, t in zip(got, want))
    for place in (g.clone(), gt.clone()):
        args = (place, gt) if torch.equal(place, g) else (g, place)
        got = E.e3conv_rms_norm_backward(want[1], w, 1, want[2], *args, grad_x=place)
        assert all(torch.equal(s, t) for s, t in zip(got, back))


def test_rows_past_32_bits():
    """Rows that lie more than 2^31 elements apart."""
    import torch
    n, step, c = 1100, 1 << 21, 64
    store = torch.empty(n * step, dtype=torch.bfloat16, device="cuda").view(n, step)
    x, g = draw(1, "bf16", n, c), draw(2, "bf16", n, c)
    store[:, :c] = x
    store[:, c:2 * c] = g
    w = weight_of(c)
    y, _, rstd = E.e3conv_rms_norm(x, w)
    far = E.e3conv_rms_norm(store[:, :c], w, out=store[:, 2 * c:3 * c])[0]
    gx, gw = E.e3conv_rms_norm_backward(x, w, 1, rstd, g)
    fx, fw = E.e3conv_rms_norm_backward(store[:, :c], w, 1, rstd, store[:, c:2 * c], grad_x=store[:, 3 * c:4 * c])
    torch.cuda.synchronize()
    assert torch.equal(far, y) and torch.equal(fx, gx) and torch.equal(fw, gw)


def test_no_rows():
    import torch
    x = torch.empty((0, 16), device="cuda")
    w = weight_of(16)
    y, total, rstd = E.e3conv_rms_norm(x, w, 2, residual=x)
    assert y.shape == total.shape == (0, 16) and rstd.shape == (0, 2)
    gx, gw = E.e3conv_rms_norm_backward(x, w, 2, rstd, x)
    assert gx.shape == (0, 16) and bool((gw == 0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_function(dtype):
    """The autograd function: both results' gradients meet in x and the residual; a result may go unused."""
    import torch
    n, c = 40, 48
    leaf = lambda s: draw(s, dtype, n, c).requires_grad_()
    x, res, w = leaf(1), leaf(2), weight_of(12).requires_grad_()
    g, gt = draw(3, dtype, n, c), draw(4, dtype, n, c)
    y, total = E.RMSNormFunction.apply(x, w, 2, 1e-5, res)
    _, _, rstd = E.e3conv_rms_norm(x.detach(), w.detach(), 2, residual=res.detach())
    for gy, gs in ((g, gt), (g, None), (None, gt)):
        outs, grads = zip(*[(o, t) for o, t in ((y, gy), (total, gs)) if t is not None])
        got = torch.autograd.grad(outs, (x, res, w), grads, retain_graph=True)
        want = E.e3conv_rms_norm_backward(total.detach(), w.detach(), 2, rstd,
                                          torch.zeros_like(g) if gy is None else gy, gs)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[0]) and torch.equal(got[2], want[1])
    z = E.RMSNormFunction.apply(x, None, 3)
    gx, = torch.autograd.grad(z, x, g.t().contiguous().t())
    assert torch.equal(gx, E.e3conv_rms_norm_backward(x.detach(), None, 3, E.e3conv_rms_norm(x.detach(), None, 3)[2], g)[0])
    (E.RMSNormFunction.apply(x, w, 2, 1e-5, res)[0] * g).sum().backward()
    assert x.grad is not res.grad and torch.equal(x.grad, res.grad)
    assert x.grad.data_ptr() != res.grad.data_ptr()


def test_gradient_is_the_forwards_difference():
    """fp32 directional derivative by central differences of the library's own forward: with steps of h the
    difference errs by about 2^-24 |L| / h from rounding and h^2 from curvature."""
    import torch
    n, c, h = 64, 40, 3e-3
    x, res, d, g, gt = (draw(s, "f32", n, c).double() for s in range(5))
    w = weight_of(20)
    f = lambda t: [o.double() for o in E.e3conv_rms_norm(t.float(), w, 2, residual=res.float())[:2]]
    loss = lambda t: sum((o * q).sum() for o, q in zip(f(t), (g, gt)))
    _, total, rstd = E.e3conv_rms_norm(x.float(), w, 2, residual=res.float())
    gx, _ = E.e3conv_rms_norm_backward(total, w, 2, rstd, g.float(), gt.float())
    slope = float((loss(x + h * d) - loss(x - h * d)) / (2 * h))
    size = float((gx.double() * d).abs().sum())
    assert abs(slope - float((gx.double() * d).sum())) <= 1e-4 * size


def test_graphs_and_streams():
    """Captured and replayed between eager work, and on another stream: the eager bits every time."""
    import torch
    n, c = 3000, 256
    x, res, g, gt = (draw(s, "bf16", n, c) for s in range(4))
    w = weight_of(64)

    def step(stream=None):
        y, total, rstd = E.e3conv_rms_norm(x, w, 4, residual=res, stream=stream)
        return (y, total, rstd) + E.e3conv_rms_norm_backward(total, w, 4, rstd, g, gt, stream=stream)

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
