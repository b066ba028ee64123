"""Attention among the nodes of each graph and its reverse pass against oracle.attention.

Tolerances are the elementwise bounds of oracle.attention.bounds: fp32 roundings of
u = 2^-24, sums of n terms within 4 sqrt(n) u of their magnitudes, and for bf16 one
rounding of 2^-8 (eight significant bits) for P, for dS and for every stored result.
"""

import numpy as np
import pytest

from oracle import attention
from equivariant_gnn_message_amd import e3conv as E

from ._gpu import say

pytestmark = pytest.mark.gpu

U = {"f32": (2.0 ** -24, 0.0), "bf16": (2.0 ** -24, 2.0 ** -8)}


def ptr(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def dtype_of(name):
    import torch
    return torch.float32 if name == "f32" else torch.bfloat16


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.detach().double().cpu().numpy()


def draw(seed, dtype, lens_q, lens_k, hq, hk, d, dv, spread=1.0):
    import torch
    gen = torch.Generator().manual_seed(seed)
    nq, nk = int(sum(lens_q)), int(sum(lens_k))
    return [(spread * torch.randn(s, generator=gen)).to(dtype_of(dtype)).cuda()
            for s in ((nq, hq, d), (nk, hk, d), (nk, hk, dv), (nq, hq, dv))]


def check(dtype, q, k, v, g, lens_q, lens_k, scale=None, q_mask=None, k_mask=None, backward=True, label=""):
    import torch
    qp, kp = ptr(lens_q), ptr(lens_k)
    dqp, dkp = dev(qp), dev(kp)
    scale = q.shape[2] ** -0.5 if scale is None else scale
    masks = dict(q_mask=None if q_mask is None else dev(q_mask), k_mask=None if k_mask is None else dev(k_mask))
    say(f"[attention] {dtype} q {tuple(q.shape)} k {tuple(k.shape)} v {tuple(v.shape)} {label}")
    out, lse = E.e3conv_attention(q, k, v, dqp, dkp, scale, **masks)
    torch.cuda.synchronize()
    u, r = U[dtype]
    clean = lambda t, m: t if m is None else np.where(np.asarray(m, bool)[:, None, None], t, 0.0)
    args = (clean(host(q), q_mask), clean(host(k), k_mask), clean(host(v), k_mask), qp, kp, np.float32(scale), u, r,
            q_mask, k_mask)
    want, tol = attention.bounds(*args, grad=clean(host(g), q_mask) if backward else None)
    got = {"out": host(out), "lse": host(lse)}
    if backward:
        gq, gk, gv = E.e3conv_attention_backward(q, k, v, out, lse, g, dqp, dkp, scale, **masks)
        torch.cuda.synchronize()
        got.update(dq=host(gq), dk=host(gk), dv=host(gv))
    for name in got:
        a, b = got[name], want[name]
        same = np.isneginf(a) & np.isneginf(b)
        off = np.abs(np.where(same, 0.0, a) - np.where(same, 0.0, b))
        assert np.all(np.isfinite(off)), name
        worst = float(np.max(off - tol[name], initial=-1.0))
        say(f"  {name}: max err {float(np.max(off, initial=0.0)):.3e}, over its bound by {worst:.3e}")
        assert worst <= 1e-30, (name, worst)
    return got


LENS = [0, 1, 2, 63, 64, 65, 130, 257]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk,d,dv", [(1, 1, 1, 1), (2, 2, 8, 8), (3, 1, 33, 20), (4, 2, 64, 64), (4, 4, 32, 96),
                                        (8, 2, 16, 128), (2, 1, 100, 100), (2, 2, 128, 128), (5, 5, 48, 7)])
def test_self_attention(dtype, hq, hk, d, dv):
    check(dtype, *draw(d + dv, dtype, LENS, LENS, hq, hk, d, dv), LENS, LENS)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens_q,lens_k", [
    ([1], [1]), ([1], [700]), ([1, 1, 1], [50, 0, 3]), ([0, 4], [9, 0]), ([700], [1]), ([3, 0, 300], [5, 40, 64]),
    ([2, 1], [3000, 1]), ([513], [129])], ids=str)
def test_cross_attention(dtype, lens_q, lens_k):
    for heads in ((1, 1), (8, 2), (6, 6)):
        check(dtype, *draw(7, dtype, lens_q, lens_k, *heads, 64, 64), lens_q, lens_k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_axis_of_few_rows(dtype):
    """One query over many keys, and many queries over one key: split axes, joined."""
    for lens_q, lens_k in (([1], [70001]), ([3, 2], [20011, 301]), ([30011], [1]), ([9001], [5])):
        check(dtype, *draw(3, dtype, lens_q, lens_k, 4, 2, 40, 24), lens_q, lens_k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [16, 33, 64, 128])
def test_masked_nodes_hold_anything(dtype, d):
    """NaN and infinities in masked rows reach nothing; graphs without a seen key give zeros."""
    import torch
    lens = [70, 5, 129, 0, 64]
    q, k, v, g = draw(11, dtype, lens, lens, 4, 2, d, d)
    rng = np.random.default_rng(5)
    mask = (rng.random(sum(lens)) < 0.7).astype(np.uint8)
    mask[70:75] = 0                       # a graph of padding alone
    mask[75:75 + 64] = 0                  # whole tiles of padding
    hole = torch.from_numpy(mask == 0).cuda()
    for t, bad in ((q, float("nan")), (k, float("inf")), (v, float("nan")), (g, float("nan"))):
        t[hole] = bad
    got = check(dtype, q, k, v, g, lens, lens, q_mask=mask, k_mask=mask)
    for name in ("out", "dq", "dk", "dv"):
        assert np.all(got[name][mask == 0] == 0)
    assert np.all(np.isneginf(got["lse"][mask == 0]))
    # bool masks, and a mask of the keys alone
    import torch
    b = torch.from_numpy(mask != 0).cuda()
    out, _ = E.e3conv_attention(q, k, v, dev(ptr(lens)), dev(ptr(lens)), None, b, b)
    np.testing.assert_array_equal(host(out), got["out"])
    q, k, v, g = draw(12, dtype, lens, lens, 4, 2, d, d)
    k[hole], v[hole] = float("nan"), float("-inf")
    got = check(dtype, q, k, v, g, lens, lens, k_mask=mask)
    assert np.all(got["out"][70:75] == 0) and np.all(got["dq"][70:75] == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_logits(dtype):
    """Logits of some hundreds: the maximum is subtracted, one key takes the weight."""
    lens = [65, 130]
    check(dtype, *draw(21, dtype, lens, lens, 2, 2, 64, 64, spread=4.0), lens, lens, scale=1.0)
    check(dtype, *draw(22, dtype, lens, lens, 2, 1, 64, 64), lens, lens, scale=-0.3)
    check(dtype, *draw(23, dtype, lens, lens, 2, 1, 64, 64), lens, lens, scale=0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_inputs_average(dtype):
    """Zero queries: every seen key has the same probability, lse = log of their number."""
    import torch
    lens = [0, 1, 77]
    q, k, v, g = draw(31, dtype, lens, lens, 1, 1, 16, 16)
    q.zero_()
    out, lse = E.e3conv_attention(q, k, v, dev(ptr(lens)), dev(ptr(lens)))
    torch.cuda.synchronize()
    np.testing.assert_allclose(host(lse)[1:, 0], np.log(77), rtol=1e-6)
    assert host(lse)[0, 0] == 0 and np.array_equal(host(out)[0], host(v)[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides_and_alignment(dtype):
    """Packed projections, heads-first storage, unaligned rows, a repeated (zero-stride) operand, and
    gradients written into strided storage: bit-equal to the dense call."""
    import torch
    lens = [33, 0, 100]
    n, p = sum(lens), dev(ptr(lens))
    q, k, v, g = draw(41, dtype, lens, lens, 4, 2, 24, 24)
    ref, lse = E.e3conv_attention(q, k, v, p, p)
    grads = E.e3conv_attention_backward(q, k, v, ref, lse, g, p, p)
    packed = torch.cat([q, k, v], 1)                                 # (n, 8, 24)
    first = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # heads first in memory

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:]
        return flat.view(t.shape).copy_(t)

    odd = lambda t: torch.cat([t, t[..., :1]], 2)[..., :24]            # rows of 25
    for name, (a, b, c) in {"packed": (packed[:, :4], packed[:, 4:6], packed[:, 6:]),
                            "heads first": (first(q), first(k), first(v)),
                            "shifted": (shifted(q), shifted(k), shifted(v)),
                            "odd rows": (odd(q), odd(k), odd(v))}.items():
        say(f"[attention] {dtype} strides: {name}")
        out, l2 = E.e3conv_attention(a, b, c, p, p)
        got = E.e3conv_attention_backward(a, b, c, first(out), l2, odd(g), p, p)
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(l2, lse), name
        for x, y in zip(got, grads):
            assert torch.equal(x, y), name
    store = torch.full((n, 9, 24), 7.0, dtype=q.dtype, device="cuda")
    into = (store[:, :4], store[:, 4:6], store[:, 6:8])
    E.e3conv_attention_backward(q, k, v, ref, lse, g, p, p, grads=into)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(into, grads)) and bool((store[:, 8] == 7).all())
    out = torch.full((n, 5, 24), 7.0, dtype=q.dtype, device="cuda")
    E.e3conv_attention(q, k, v, p, p, out=out[:, :4])
    torch.cuda.synchronize()
    assert torch.equal(out[:, :4], ref) and bool((out[:, 4] == 7).all())
    one = k[:, :1].expand(n, 4, 24)                                  # one key head repeated
    a = E.e3conv_attention(q, one, one, p, p)[0]
    b = E.e3conv_attention(q, one.contiguous(), one.contiguous(), p, p)[0]
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Rows that lie more than 2^31 elements apart in a long cache."""
    import torch
    nk, step = 1100, 1 << 21
    store = torch.empty(nk * step, dtype=torch.bfloat16, device="cuda")
    q, k, v, g = draw(51, "bf16", [3], [nk], 1, 1, 64, 64)
    rows = store.view(nk, 1, step)
    fk, fv = rows[:, :, :64], rows[:, :, 64:128]
    fk.copy_(k)
    fv.copy_(v)
    gk, gv = rows[:, :, 128:192], rows[:, :, 192:256]
    a, b = dev(ptr([3])), dev(ptr([nk]))
    ref, lse = E.e3conv_attention(q, k, v, a, b)
    out, _ = E.e3conv_attention(q, fk, fv, a, b)
    want = E.e3conv_attention_backward(q, k, v, ref, lse, g, a, b)
    got = E.e3conv_attention_backward(q, fk, fv, ref, lse, g, a, b, grads=(torch.empty_like(q), gk, gv))
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_every_time_and_on_other_streams(dtype):
    import torch
    lens = [300, 1, 513]
    q, k, v, g = draw(61, dtype, lens, lens, 4, 2, 64, 64)
    p = dev(ptr(lens))

    def step(stream=None):
        out, lse = E.e3conv_attention(q, k, v, p, p, stream=stream)
        return (out, lse) + E.e3conv_attention_backward(q, k, v, out, lse, g, p, p, stream=stream)

    ref = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        for _ in range(3):
            got = step(stream)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_graph_replays():
    """Captured once, replayed with eager work between: every replay equals the eager result."""
    import torch
    lens_q, lens_k = [40, 3, 200], [40, 5000, 200]
    q, k, v, g = draw(71, "bf16", lens_q, lens_k, 4, 2, 64, 64)
    a, b = dev(ptr(lens_q)), dev(ptr(lens_k))
    out, lse = E.e3conv_attention(q, k, v, a, b)
    grads = E.e3conv_attention_backward(q, k, v, out, lse, g, a, b)
    ref = [t.clone() for t in (out, lse) + grads]

    def step():
        E.e3conv_attention(q, k, v, a, b, out=out, lse=lse)
        E.e3conv_attention_backward(q, k, v, out, lse, g, a, b, grads=grads)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        for t in (out, lse) + grads:
            t.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((out, lse) + grads, ref))


def test_autograd_and_shared_heads():
    """AttentionFunction: gradients of an expanded (repeated) key head sum over its copies, and a
    directional difference of the loss agrees (h = 1/64: truncation h^2/6 of an O(10) third derivative
    and rounding of a sum of ~6000 terms of fp32 over h, both below 1e-2 of the slope's scale)."""
    import torch
    lens = [20, 0, 33]
    p = dev(ptr(lens))
    q, k, v, g = draw(81, "f32", lens, lens, 4, 1, 16, 16)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    F = E.AttentionFunction

    def loss(a, b, c):
        return (F.apply(a, b.expand(-1, 4, -1), c, p, p) * g).sum()

    loss(leaves[0], leaves[1], leaves[2].expand(-1, 4, -1)).backward()
    out, lse = E.e3conv_attention(q, k, v, p, p)
    want = E.e3conv_attention_backward(q, k, v, out, lse, g, p, p)
    for t, w in zip(leaves, want):
        torch.testing.assert_close(t.grad, w, rtol=1e-4, atol=1e-5)
    gen = torch.Generator().manual_seed(3)
    way = [torch.randn(t.shape, generator=gen).cuda() for t in (q, k, v)]
    at = lambda h: float((F.apply(*(t + h * w for t, w in zip((q, k, v), way)), p, p).double() * g.double()).sum())
    slope = sum(float((t.grad.double() * w.double()).sum()) for t, w in zip(leaves, way))
    h = 1 / 64
    diff = (8 * (at(h) - at(-h)) - (at(2 * h) - at(-2 * h))) / (12 * h)
    scale = sum(float((t.grad.double().norm() * 1.0)) for t in leaves)
    assert abs(diff - slope) <= 1e-2 * scale, (diff, slope, scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens_q,lens_k", [([300], [2000]), ([577, 40], [527, 1500]), ([2247], [2247])], ids=str)
def test_rows_and_keys_split_in_few(dtype, lens_q, lens_k):
    """Too few row tiles to fill the device, but many rows: a few splits, joined element by element."""
    mask = (np.random.default_rng(9).random(sum(lens_k)) < 0.9).astype(np.uint8)
    check(dtype, *draw(111, dtype, lens_q, lens_k, 4, 2, 24, 40), lens_q, lens_k, k_mask=mask)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,dv", [(16, 16), (33, 20), (64, 64), (100, 128)])
def test_many_small_graphs(dtype, d, dv):
    """Graphs of at most 64 rows on average take one launch for the whole reverse pass; one of them is much longer."""
    lens = [5, 0, 64, 1, 33, 64, 200, 17, 2, 63] * 2
    rng = np.random.default_rng(8)
    mask = (rng.random(sum(lens)) < 0.8).astype(np.uint8)
    check(dtype, *draw(101, dtype, lens, lens, 4, 4, d, dv), lens, lens, q_mask=mask, k_mask=mask)
    some = [1, 3, 0, 2, 4, 1, 2, 0, 1, 1] * 2
    check(dtype, *draw(102, dtype, some, lens, 4, 2, d, dv), some, lens, k_mask=mask)
    check(dtype, *draw(103, dtype, lens, some, 1, 1, d, dv), lens, some)


def test_empty_calls():
    import torch
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    e = torch.empty((0, 2, 8), device="cuda")
    out, lse = E.e3conv_attention(e, e, e, z, z)
    assert out.shape == (0, 2, 8) and lse.shape == (0, 2)
    # keys without queries: zero gradients; queries without keys: zeros and -inf
    n = torch.ones((3, 2, 8), device="cuda")
    a, b = dev(ptr([0])), dev(ptr([3]))
    o, l = E.e3conv_attention(e, n, n, a, b)
    gq, gk, gv = E.e3conv_attention_backward(e, n, n, o, l, e, a, b)
    assert not gk.any() and not gv.any() and gq.shape == (0, 2, 8)
    o, l = E.e3conv_attention(n, e, e, b, a)
    gq, gk, gv = E.e3conv_attention_backward(n, e, e, o, l, n, b, a)
    assert not o.any() and bool(torch.isneginf(l).all()) and not gq.any()


def test_refusals_on_device():
    import torch
    lens = [4]
    q, k, v, g = draw(91, "f32", lens, lens, 2, 2, 8, 8)
    p = dev(ptr(lens))
    out, lse = E.e3conv_attention(q, k, v, p, p)
    lq, lk, lv, lg = draw(92, "f32", [9000], [9000], 2, 2, 8, 8)
    lp = dev(ptr([9000]))
    lout, llse = E.e3conv_attention(lq, lk, lv, lp, lp)
    for err, call in (
            (TypeError, lambda: E.e3conv_attention(q, k.bfloat16(), v, p, p)),
            (TypeError, lambda: E.e3conv_attention(q.half(), k.half(), v.half(), p, p)),
            (ValueError, lambda: E.e3conv_attention(q, k[:3], v, p, p)),
            (ValueError, lambda: E.e3conv_attention(q, k.transpose(1, 2).contiguous().transpose(1, 2), v, p, p)),
            (TypeError, lambda: E.e3conv_attention(q, k, v, p.long(), p)),
            (ValueError, lambda: E.e3conv_attention(q, k, v, p, p[:1])),
            (ValueError, lambda: E.e3conv_attention(q, k, v, p, p, k_mask=torch.ones(3, dtype=torch.uint8, device="cuda"))),
            (ValueError, lambda: E.e3conv_attention(q, k, v, p, p, out=q[:, :1].expand(4, 2, 8))),
            (ValueError, lambda: E.e3conv_attention(q, k.cpu(), v, p, p)),
            (E.E3ConvError, lambda: E.e3conv_attention(q, k, v, p, p, scale=float("inf"))),
            (E.E3ConvError, lambda: E.e3conv_attention(q.expand(4, 2, 8)[:, :1].repeat(1, 3, 1), k, v, p, p)),
            (E.E3ConvError, lambda: E.e3conv_attention_backward(
                lq, lk, lv, lout, llse, lg, lp, lp, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")))):
        with pytest.raises(err):
            call()
