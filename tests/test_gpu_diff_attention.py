"""Differential attention among the nodes of each graph and its reverse pass against oracle.diff_attention.

Tolerances are the elementwise bounds of oracle.diff_attention.bounds: fp32 roundings of u = 2^-24, sums of n
terms within 4 sqrt(n) u of their magnitudes, and for bf16 one rounding of 2^-8 for each map's P, for their
difference, for both dS and for every stored result.
"""

import numpy as np
import pytest

from oracle import diff_attention
from equivariant_gnn_message_amd import e3conv as E

from ._gpu import say
from .test_gpu_attention import U, dev, dtype_of, host, ptr

pytestmark = pytest.mark.gpu


def draw(seed, dtype, lens_q, lens_k, hq, hk, d, dv, spread=1.0):
    """q, k, v, lam, grad_out."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    nq, nk = int(sum(lens_q)), int(sum(lens_k))
    q, k, v, g = [(spread * torch.randn(s, generator=gen)).to(dtype_of(dtype)).cuda()
                  for s in ((nq, 2 * hq, d), (nk, 2 * hk, d), (nk, hk, dv), (nq, hq, dv))]
    return q, k, v, torch.randn(hq, generator=gen).cuda(), g


def check(dtype, q, k, v, lam, g, lens_q, lens_k, scale=None, q_mask=None, k_mask=None, backward=True, label=""):
    import torch
    qp, kp = ptr(lens_q), ptr(lens_k)
    dqp, dkp = dev(qp), dev(kp)
    scale = q.shape[2] ** -0.5 if scale is None else scale
    masks = dict(q_mask=None if q_mask is None else dev(q_mask), k_mask=None if k_mask is None else dev(k_mask))
    say(f"[diff] {dtype} q {tuple(q.shape)} k {tuple(k.shape)} v {tuple(v.shape)} {label}")
    out, second, lse = E.e3conv_diff_attention(q, k, v, lam, dqp, dkp, scale, **masks)
    torch.cuda.synchronize()
    u, r = U[dtype]
    clean = lambda t, m: host(t) if m is None else np.where(np.asarray(m, bool)[:, None, None], host(t), 0.0)
    want, tol = diff_attention.bounds(clean(q, q_mask), clean(k, k_mask), clean(v, k_mask), host(lam), qp, kp,
                                      np.float32(scale), u, r, q_mask, k_mask, clean(g, q_mask) if backward else None)
    got = {"out": host(out), "second": host(second), "lse": host(lse)}
    if backward:
        grads = E.e3conv_diff_attention_backward(q, k, v, lam, out, second, lse, g, dqp, dkp, scale, **masks)
        torch.cuda.synchronize()
        got.update(zip(("dq", "dk", "dv", "dlam"), map(host, grads)))
    for name in got:
        a, b = got[name], want[name]
        same = np.isneginf(a) & np.isneginf(b)
        off = np.abs(np.where(same, 0.0, a) - np.where(same, 0.0, b))
        assert np.all(np.isfinite(off)), name
        worst = float(np.max(off - tol[name], initial=-1.0))
        say(f"  {name}: max err {float(np.max(off, initial=0.0)):.3e}, over its bound by {worst:.3e}")
        assert worst <= 1e-30, (name, worst)
    return got


LENS = [0, 1, 2, 31, 32, 33, 64, 65, 130, 257]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk,d,dv", [(1, 1, 1, 1), (1, 1, 16, 32), (2, 2, 8, 16), (3, 1, 33, 20), (4, 2, 64, 128),
                                        (4, 4, 32, 64), (8, 2, 16, 128), (2, 1, 50, 100), (2, 2, 64, 64), (5, 5, 24, 7),
                                        (6, 2, 40, 80), (2, 1, 32, 40)])
def test_self_attention(dtype, hq, hk, d, dv):
    check(dtype, *draw(d + dv, dtype, LENS, LENS, hq, hk, d, dv), LENS, LENS)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens_q,lens_k", [
    ([1], [1]), ([1], [700]), ([1, 1, 1], [50, 0, 3]), ([0, 4], [9, 0]), ([700], [1]), ([3, 0, 300], [5, 40, 64]),
    ([2, 1], [3000, 1]), ([513], [129])], ids=str)
def test_cross_attention(dtype, lens_q, lens_k):
    for heads, d, dv in (((1, 1), 64, 128), ((8, 2), 32, 64), ((6, 6), 64, 128)):
        check(dtype, *draw(7, dtype, lens_q, lens_k, *heads, d, dv), lens_q, lens_k)


def means_bound(q, k, v, lam, g, scale, u, r, out, second):
    """dq of one graph (heads of q and k alike) in 64 bits from out and second as given, and how far it may be off.

    Roundings of the keys are independent, so a sum of n of them is within four times the root of their squares:
    dS by r; P by its logits' rounding and dP by its dot product's, 4 sqrt(dims) u of their magnitudes; the running
    sum by u of its size in every step.  The row's own errors scale dq: lse's and the result's rounding.  What
    the deltas of out and second are off is taken off again, up to B's rounding, by 2^-8 whatever the type, and
    to the rounding of r's sum; it does not stand here times B itself.
    """
    want, tol = np.zeros_like(q), np.zeros_like(q)
    n, dims = len(k), 4 * np.sqrt(max(q.shape[2], v.shape[2]))
    for h in range(len(lam)):
        dp = g[:, h] @ v[:, h].T
        size = np.abs(g[:, h]) @ np.abs(v[:, h]).T
        d1 = (g[:, h] * second[:, h]).sum(1, keepdims=True)
        d0 = (g[:, h] * out[:, h]).sum(1, keepdims=True) + lam[h] * d1
        for m, given, f in ((0, d0, 1.0), (1, d1, -lam[h])):
            qh, kh = q[:, 2 * h + m], k[:, 2 * h + m]
            s = scale * qh @ kh.T
            top = s.max(1, keepdims=True)
            lse = top + np.log(np.exp(s - top).sum(1, keepdims=True))
            p = np.exp(s - lse)
            delta = (p * dp).sum(1, keepdims=True)
            ds = p * (dp - delta)
            a = abs(scale * f)
            want[:, 2 * h + m] = scale * f * ds @ kh
            logit = u * (dims * scale * (np.abs(qh) @ np.abs(kh).T) + 4 * np.abs(s) + 4 * np.abs(top) + 8)
            each = (r + logit) * np.abs(ds) + p * u * (dims * size + 4 * (np.abs(dp) + np.abs(delta)))
            row = logit.max(1, keepdims=True) + 4 * u * (np.abs(lse) + np.sqrt(n))
            sums = 4 * np.sqrt(n) * u * 4 * np.sqrt(ds ** 2 @ kh ** 2)
            rest = np.abs(given - delta)
            left = (4 * np.sqrt(n) * u * (p * np.abs(dp - given)).sum(1, keepdims=True) * np.abs(p @ kh)
                    + rest * 4 * 2.0 ** -8 * np.sqrt(p ** 2 @ kh ** 2) + rest * (4 * np.sqrt(n) + 8) * u * (p @ np.abs(kh)))
            tol[:, 2 * h + m] = a * (4 * np.sqrt(each ** 2 @ kh ** 2) + sums + left) \
                + (r + row) * np.abs(want[:, 2 * h + m])
    return want, tol


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,keys,heads,d,dv", [(2500, 2500, 2, 32, 64), (2500, 2500, 1, 64, 128), (3, 20011, 2, 64, 128),
                                                  (70, 3001, 2, 33, 40), (50, 900, 1, 16, 32)])
def test_gradient_of_q_where_v_has_a_mean(dtype, rows, keys, heads, d, dv):
    """Long graphs, v and grad_out of mean 2: what out and second lose in their roundings is off delta by a multiple of
    what the keys' own terms differ by, and is not in grad_q."""
    import torch
    gen = torch.Generator().manual_seed(rows + d)
    q, k, v, g = [(mean + torch.randn(s, generator=gen)).to(dtype_of(dtype)).cuda() for mean, s in (
        (0.0, (rows, 2 * heads, d)), (0.0, (keys, 2 * heads, d)), (2.0, (keys, heads, dv)), (2.0, (rows, heads, dv)))]
    lam = torch.linspace(0.3, 0.8, heads).cuda()
    qp, kp = dev(ptr([rows])), dev(ptr([keys]))
    say(f"[diff means] {dtype} {rows} x {keys} heads {heads} {d} {dv}")
    out, second, lse = E.e3conv_diff_attention(q, k, v, lam, qp, kp)
    grads = E.e3conv_diff_attention_backward(q, k, v, lam, out, second, lse, g, qp, kp)
    torch.cuda.synchronize()
    u, r = U[dtype]
    want, tol = means_bound(*map(host, (q, k, v, lam, g)), float(np.float32(d ** -0.5)), u, r, host(out), host(second))
    off = np.abs(host(grads[0]) - want)
    worst = float(np.max(off / tol))
    say(f"  dq: max err {off.max():.3e}, {worst:.2f} of its bound")
    assert worst <= 1.0

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_axis_of_few_rows(dtype):
    """One query over many keys, and many queries over one key: split axes, joined."""
    for lens_q, lens_k in (([1], [70001]), ([3, 2], [20011, 301]), ([30011], [1]), ([9001], [5])):
        check(dtype, *draw(3, dtype, lens_q, lens_k, 4, 2, 40, 24), lens_q, lens_k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads", [(40, 1), (200, 2), (300, 1)])
def test_many_heads_share(dtype, heads):
    """More query heads of a kv head than a tile has rows."""
    lens_q, lens_k = [3, 0, 5, 1], [40, 3, 0, 70]
    check(dtype, *draw(5, dtype, lens_q, lens_k, *heads, 16, 32), lens_q, lens_k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,dv", [(16, 32), (33, 48), (32, 64), (64, 128), (40, 100)])
def test_masked_nodes_hold_anything(dtype, d, dv):
    """NaN and infinities in masked rows reach nothing; graphs without a seen key give zeros."""
    import torch
    lens = [70, 5, 129, 0, 64]
    q, k, v, lam, g = draw(11, dtype, lens, lens, 4, 2, d, dv)
    rng = np.random.default_rng(5)
    mask = (rng.random(sum(lens)) < 0.7).astype(np.uint8)
    mask[70:75] = 0                       # a graph of padding alone
    mask[75:75 + 64] = 0                  # whole tiles of padding
    hole = torch.from_numpy(mask == 0).cuda()
    for t, bad in ((q, float("nan")), (k, float("inf")), (v, float("nan")), (g, float("nan"))):
        t[hole] = bad
    got = check(dtype, q, k, v, lam, g, lens, lens, q_mask=mask, k_mask=mask)
    for name in ("out", "second", "dq", "dk", "dv"):
        assert np.all(got[name][mask == 0] == 0)
    assert np.all(np.isneginf(got["lse"][mask == 0]))
    b = torch.from_numpy(mask != 0).cuda()
    out, _, _ = E.e3conv_diff_attention(q, k, v, lam, dev(ptr(lens)), dev(ptr(lens)), None, b, b)
    np.testing.assert_array_equal(host(out), got["out"])
    q, k, v, lam, g = draw(12, dtype, lens, lens, 4, 2, d, dv)
    k[hole], v[hole] = float("nan"), float("-inf")
    got = check(dtype, q, k, v, lam, g, lens, lens, k_mask=mask)
    assert np.all(got["out"][70:75] == 0) and np.all(got["dq"][70:75] == 0)
    none = np.zeros(sum(lens), np.uint8)
    got = check(dtype, *draw(13, dtype, lens, lens, 4, 2, d, dv), lens, lens, k_mask=none)
    assert np.all(got["dlam"] == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_logits(dtype):
    """Logits of some hundreds: the maximum of each map is subtracted, one key takes the weight."""
    lens = [65, 130]
    check(dtype, *draw(21, dtype, lens, lens, 2, 2, 64, 64, spread=4.0), lens, lens, scale=1.0)
    check(dtype, *draw(22, dtype, lens, lens, 2, 1, 64, 64), lens, lens, scale=-0.3)
    check(dtype, *draw(23, dtype, lens, lens, 2, 1, 32, 64), lens, lens, scale=0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,dv", [(32, 64), (64, 128)])
def test_weights_of_the_second_map(dtype, d, dv):
    """lambda of 0 is the plain attention of the first map; of 1 with equal maps nothing is left; large and negative."""
    import torch
    lens = [65, 130, 1]
    p = dev(ptr(lens))
    q, k, v, lam, g = draw(31, dtype, lens, lens, 4, 2, d, dv)
    lam = torch.tensor([0.0, 1.0, -30.0, 100.0], device="cuda")
    check(dtype, q, k, v, lam, g, lens, lens)
    first, _ = E.e3conv_attention(q[:, 0::2], k[:, 0::2], v, p, p)
    out, second, _ = E.e3conv_diff_attention(q, k, v, torch.zeros_like(lam), p, p)
    other, _ = E.e3conv_attention(q[:, 1::2], k[:, 1::2], v, p, p)
    # two evaluations, each of the oracle's accuracy: a result's rounding and those of P, averaged
    tol = dict(rtol=2.0 ** -7, atol=2.0 ** -7) if dtype == "bf16" else dict(rtol=1e-5, atol=1e-5)
    torch.testing.assert_close(out, first, **tol)
    torch.testing.assert_close(second, other, **tol)
    same = lambda t: t[:, 0::2].repeat_interleave(2, 1)
    out, _, _ = E.e3conv_diff_attention(same(q), same(k), v, torch.ones_like(lam), p, p)
    assert bool((out == 0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,dv", [(24, 40), (32, 64), (64, 128)])
def test_strides_and_alignment(dtype, d, dv):
    """Packed projections, heads first, unaligned and odd rows, a repeated operand, gradients and results in wider
    storage: bit-equal to the dense call, or as near as another order of loads leaves them."""
    import torch
    lens = [33, 0, 100]
    n, p = sum(lens), dev(ptr(lens))
    q, k, v, lam, g = draw(41, dtype, lens, lens, 4, 2, d, dv)
    ref = E.e3conv_diff_attention(q, k, v, lam, p, p)
    grads = E.e3conv_diff_attention_backward(q, k, v, lam, *ref, g, p, p)
    packed = torch.cat([q, k], 1)                                     # (n, 12, d)
    first = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # heads first in memory

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:]
        return flat.view(t.shape).copy_(t)

    odd = lambda t: torch.cat([t, t[..., :1]], 2)[..., :t.shape[2]]
    for name, (a, b, c) in {"packed": (packed[:, :8], packed[:, 8:], v), "heads first": (first(q), first(k), first(v)),
                            "shifted": (shifted(q), shifted(k), shifted(v)), "odd rows": (odd(q), odd(k), odd(v))}.items():
        say(f"[diff] {dtype} strides: {name}")
        got = E.e3conv_diff_attention(a, b, c, lam, p, p)
        back = E.e3conv_diff_attention_backward(a, b, c, lam, first(got[0]), odd(got[1]), got[2], odd(g), p, p)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, ref)), name
        assert all(torch.equal(x, y) for x, y in zip(back, grads)), name
    wide = torch.full((n, 15, max(d, dv)), 7.0, dtype=q.dtype, device="cuda")
    into = (wide[:, :8, :d], wide[:, 8:12, :d], wide[:, 12:14, :dv])
    E.e3conv_diff_attention_backward(q, k, v, lam, *ref, g, p, p, grads=into)
    assert all(torch.equal(x, y) for x, y in zip(into, grads)) and bool((wide[:, 14] == 7).all())
    wide = torch.full((n, 9, dv), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.empty_like(ref[2])
    E.e3conv_diff_attention(q, k, v, lam, p, p, out=wide[:, :4], second=wide[:, 4:8], lse=lse)
    assert torch.equal(wide[:, :4], ref[0]) and torch.equal(wide[:, 4:8], ref[1]) and torch.equal(lse, ref[2])
    assert bool((wide[:, 8] == 7).all())
    out, second, lse = E.e3conv_diff_attention(q, k, v, lam, p, p, keep=False)
    assert torch.equal(out, ref[0]) and second is None and lse is None
    one, va = k[:, :2].repeat(1, 2, 1), v[:, :1]
    a = E.e3conv_diff_attention(q, one, va.expand(n, 2, dv), lam, p, p)[0]
    assert torch.equal(a, E.e3conv_diff_attention(q, one, va.expand(n, 2, dv).contiguous(), lam, p, p)[0])


def test_offsets_past_32_bits():
    """Rows that lie more than 2^31 elements apart in a long cache."""
    import torch
    nk, step = 1100, 1 << 21
    store = torch.empty(nk * step, dtype=torch.bfloat16, device="cuda")
    q, k, v, lam, g = draw(51, "bf16", [3], [nk], 1, 1, 64, 128)
    rows = store.view(nk, step)
    fk, gk = (rows[:, i:i + 128].unflatten(1, (2, 64)) for i in (0, 256))
    fv, gv = (rows[:, i:i + 128].unflatten(1, (1, 128)) for i in (128, 384))
    fk.copy_(k)
    fv.copy_(v)
    a, b = dev(ptr([3])), dev(ptr([nk]))
    ref = E.e3conv_diff_attention(q, k, v, lam, a, b)
    out = E.e3conv_diff_attention(q, fk, fv, lam, a, b)
    want = E.e3conv_diff_attention_backward(q, k, v, lam, *ref, g, a, b)
    got = E.e3conv_diff_attention_backward(q, fk, fv, lam, *ref, g, a, b, grads=(torch.empty_like(q), gk, gv))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, ref)) and all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("d,dv", [(32, 64), (64, 128), (20, 33)])
def test_offsets_that_are_no_offsets(d, dv):
    """Offsets that decrease, start past 0 or leave the tensors: no access out of range, so the rest of memory stays."""
    import torch
    n = 200
    q, k, v, lam, g = draw(55, "bf16", [n], [n], 2, 1, d, dv)
    for offsets in ([5, 150, 60, 200], [-7, 90, 400, 200], [0, 200, 200, 100], [200, 0, 0, 200]):
        p = dev(np.array(offsets, np.int32))
        out = E.e3conv_diff_attention(q, k, v, lam, p, p)
        E.e3conv_diff_attention_backward(q, k, v, lam, *out, g, p, p)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_every_time_captured_and_on_other_streams(dtype):
    import torch
    lens = [300, 1, 513]
    q, k, v, lam, g = draw(61, dtype, lens, lens, 4, 2, 64, 128)
    p = dev(ptr(lens))

    def step(stream=None):
        out = E.e3conv_diff_attention(q, k, v, lam, p, p, stream=stream)
        return out + E.e3conv_diff_attention_backward(q, k, v, lam, *out, g, p, p, stream=stream)

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, side.cuda_stream):
        got = step(stream)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
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
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert all(torch.equal(x, y) for x, y in zip(step(), want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_function(dtype):
    import torch
    lens = [40, 7]
    p = dev(ptr(lens))
    q, k, v, lam, g = draw(71, dtype, lens, lens, 4, 2, 16, 32)
    leaves = [t.requires_grad_() for t in (q, k, v, lam)]
    mask = dev((np.random.default_rng(1).random(47) < 0.8).astype(np.uint8))
    out = E.DiffAttentionFunction.apply(*leaves, p, p, 0.3, mask, mask)
    got = torch.autograd.grad(out, leaves, g.transpose(0, 2).contiguous().transpose(0, 2))
    plain = [t.detach() for t in leaves]
    ref = E.e3conv_diff_attention(*plain, p, p, 0.3, mask, mask)
    want = E.e3conv_diff_attention_backward(*plain, *ref, g, p, p, 0.3, mask, mask)
    assert torch.equal(out, ref[0]) and all(torch.equal(x, y) for x, y in zip(got, want))


def test_gradients_are_the_forwards_differences():
    """fp32: central differences of the library's own forward along each operand, with steps of h: curvature gives
    h^2 / 6 of third derivatives near 1, rounding about 2^-24 sqrt(values) / h."""
    import torch
    lens, h = [30, 50], 3e-3
    p = dev(ptr(lens))
    *x, g = draw(81, "f32", lens, lens, 2, 1, 16, 32)
    along = draw(82, "f32", lens, lens, 2, 1, 16, 32)[:4]
    grads = E.e3conv_diff_attention_backward(*x, *E.e3conv_diff_attention(*x, p, p), g, p, p)
    for i, (d, grad) in enumerate(zip(along, grads)):
        def loss(t):
            y = [a + t * d if i == j else a for j, a in enumerate(x)]
            return float((E.e3conv_diff_attention(*y, p, p)[0].double() * g.double()).sum())
        terms = grad.double() * d.double()
        assert abs((loss(h) - loss(-h)) / (2 * h) - float(terms.sum())) <= 1e-3 * float(terms.abs().sum())


def test_no_rows():
    import torch
    for nq, nk in ((0, 0), (0, 5), (5, 0)):
        q, k, v, lam, g = draw(1, "f32", [nq], [nk], 2, 1, 16, 32)
        a, b = dev(ptr([nq])), dev(ptr([nk]))
        out = E.e3conv_diff_attention(q, k, v, lam, a, b)
        grads = E.e3conv_diff_attention_backward(q, k, v, lam, *out, g, a, b)
        torch.cuda.synchronize()
        assert all(bool((t == 0).all()) for t in grads + out[:2])
