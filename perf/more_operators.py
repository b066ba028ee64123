"""Measured calls of the operators of a graph-transformer block with positions: rotary positions over several
axes (forward, and backward with the gradients of positions and wave vectors), differential attention among
the nodes of each graph (forward and backward), and the root-mean-square norm of rows or heads with a
residual's addition (forward and backward).

``run`` computes them in plain torch operations where ``own`` is false and through the library's entry
points where it is true, on the same inputs.  Graphs lie one after another along the node axis; ``ptr``
holds their offsets.
"""

import math
import random

import torch

own = False

F32, BF16 = "f32", "bf16"
EPS = 1e-5


# ------------------------------------------------------------------- cases ---

def _turn(name, op, dtype, rows, heads, dim, pairs, axes, layout="adjacent", mixed=False, box=50.0, masked=False,
          packed=False):
    c = {"op": op, "dtype": dtype, "rows": rows, "heads": heads, "dim": dim, "pairs": pairs, "axes": axes,
         "layout": layout, "mixed": mixed, "box": box, "masked": masked, "packed": packed}
    return dict(c, name=name) if name else c


def _differ(name, op, dtype, graphs, queries, keys, heads, kv_heads, dim, dim_v, ragged=False, masked=False):
    c = {"op": op, "dtype": dtype, "graphs": graphs, "queries": queries, "keys": keys, "heads": heads,
         "kv_heads": kv_heads, "dim": dim, "dim_v": dim_v, "ragged": ragged, "masked": masked}
    return dict(c, name=name) if name else c


def _rms(name, op, dtype, rows, channels, groups=1, period=None, spare=0, residual=False, masked=False):
    c = {"op": op, "dtype": dtype, "rows": rows, "channels": channels, "groups": groups,
         "period": period or channels, "spare": spare, "residual": residual, "masked": masked}
    return dict(c, name=name) if name else c


def listed():
    return [
        # queries and keys of one new node of each of four growing structures: the smallest call
        _turn("turn new node f32", "turn", F32, 4, 8, 16, 8, 3, packed=True),
        # queries and keys of 100 000 nodes in one projection: ten pairs for each of x, y, z, four elements as they are
        _turn("turn 100k bf16", "turn", BF16, 100000, 12, 64, 30, 3, box=400.0, masked=True, packed=True),
        # training on 20 000 nodes with learned wave vectors; the positions' gradient is part of the forces
        _turn("turn grad 20k f32", "turn_grad", F32, 20000, 8, 32, 16, 3, "halves", mixed=True),
        # one new node of each of four growing structures attends to its structure's nodes
        _differ("differ new node f32", "differ", F32, 4, 1, 48, 2, 2, 16, 32),
        # pooling of a large graph by one query token, four heads over two shared key heads
        _differ("differ readout 100k bf16", "differ", BF16, 1, 1, 100000, 4, 2, 64, 128),
        # 100 000 nodes in about a hundred graphs of unlike sizes, with padding nodes
        _differ("differ ragged 100k bf16", "differ", BF16, 100, 1000, 1000, 4, 2, 64, 128, ragged=True, masked=True),
        # training on the gate-points batch (64 graphs of 64 nodes, 32 scalar channels as one head)
        _differ("differ grad gate batch f32", "differ_grad", F32, 64, 64, 64, 1, 1, 16, 32),
        # training on the one graph of 20 000 nodes with 128 channels, in fp32: the largest call
        _differ("differ grad 20k f32", "differ_grad", F32, 1, 20000, 20000, 2, 2, 32, 64),
        # training on ragged graphs of about 1000 nodes, 50 000 in all
        _differ("differ grad ragged 50k bf16", "differ_grad", BF16, 50, 1000, 1000, 4, 2, 64, 128, ragged=True,
                masked=True),
        # the scalar channels of the gate-points batch with the block's residual
        _rms("rms gate batch f32", "rms", F32, 4096, 32, residual=True),
        # each of four attention heads of 100 000 nodes by itself, one weight for all heads
        _rms("rms heads 100k bf16", "rms", BF16, 100000, 512, 4, 128, masked=True),
        # training on 100 000 nodes of 512 channels with the residual's gradient
        _rms("rms grad 100k bf16", "rms_grad", BF16, 100000, 512, residual=True),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    dtype = rng.choice([F32, BF16])
    kind = rng.random()
    if kind < 0.3:
        dim = rng.choice([8, 16, 24, 32, 33, 48, 64, 64, 96, 128])
        axes = rng.choice([1, 2, 3, 3, 4])
        pairs = rng.choice([dim // 2, dim // 2 // axes * axes, rng.randint(1, dim // 2)]) or 1
        heads = rng.randint(1, 24)
        while True:
            rows = _spread(rng, 1, 200000)
            if rows * heads * dim <= 1e8:
                break
        return _turn(None, rng.choice(["turn", "turn_grad"]), dtype, rows, heads, dim, pairs, axes,
                     rng.choice(["adjacent", "adjacent", "halves"]), rng.random() < 0.4,
                     float(_spread(rng, 1, 10000)), rng.random() < 0.3, rng.random() < 0.5)
    if kind < 0.7:
        op = rng.choice(["differ", "differ_grad"])
        dim = rng.choice([8, 16, 24, 32, 32, 40, 48, 64, 64, 64])
        dim_v = rng.choice([2 * dim, 2 * dim, 2 * dim, dim, rng.choice([16, 33, 64, 100, 128])])
        kv_heads = rng.choice([1, 2, 4])
        heads = kv_heads * rng.choice([1, 1, 2, 4])
        shape = rng.random()
        while True:
            graphs = _spread(rng, 1, 128)
            keys = _spread(rng, 2, 20000)
            queries = keys if shape < 0.6 else rng.randint(1, 8) if shape < 0.85 else _spread(rng, 1, 4000)
            pairs = graphs * queries * keys * heads * 1.25
            rows = graphs * max(queries * heads, keys * kv_heads) * (4 * dim + 2 * dim_v)
            if pairs <= 7e8 and pairs * dim <= 2.5e10 and rows <= 1.5e8:
                break
        return _differ(None, op, dtype, graphs, queries, keys, heads, kv_heads, dim, dim_v,
                       graphs > 3 and rng.random() < 0.5, rng.random() < 0.4)
    # rows of channels, heads that share a weight, or an l-block's components that share it
    width = rng.choice([7, 8, 16, 24, 32, 48, 64, 72, 128, 200, 256, 512, 1024, 2048])
    form = rng.choice(["rows", "rows", "heads", "block"])
    n = 1 if form == "rows" else rng.choice([2, 4, 8, 12]) if form == "heads" else rng.choice([3, 5, 7])
    while True:
        rows = _spread(rng, 1, 400000)
        if rows * width * n <= 6e7:
            break
    return _rms(None, rng.choice(["rms", "rms_grad"]), dtype, rows, width * n, n if form == "heads" else 1, width,
                rng.choice([0, 0, width]), rng.random() < 0.5, rng.random() < 0.3)


def _lengths(graphs, mean, ragged):
    """Nodes of each graph; among unlike ones a graph of one node and one of none."""
    if not ragged:
        return [mean] * graphs
    r = random.Random(graphs * 1000003 + mean)
    n = [max(1, int(mean * r.uniform(0.5, 1.5))) for _ in range(graphs)]
    n[1], n[2] = 1, 0
    return n


def _lengths_of(c):
    k = _lengths(c["graphs"], c["keys"], c["ragged"])
    q = k if c["queries"] == c["keys"] else _lengths(c["graphs"], c["queries"], c["ragged"])
    return q, k


def work(case):
    size = 4 if case["dtype"] == F32 else 2
    op = case["op"]
    if op.startswith("turn"):
        n, angles = case["rows"] * case["heads"], case["rows"] * case["pairs"]
        tensors, per = (2, 6) if op == "turn" else (3, 9)
        fixed = 4 * case["rows"] * case["axes"] * (1 if op == "turn" else 2)
        return {"bytes": tensors * n * case["dim"] * size + fixed,
                "flops": per * n * case["pairs"] + (2 * case["axes"] + 2) * angles}
    if op.startswith("rms"):
        n = case["rows"] * case["channels"]
        tensors = 2 + 2 * case["residual"] if op == "rms" else 3 + case["residual"]
        return {"bytes": tensors * n * size + 4 * case["rows"] * case["groups"],
                "flops": (5 if op == "rms" else 9) * n}
    lq, lk = _lengths_of(case)
    pairs = sum(a * b for a, b in zip(lq, lk)) * case["heads"]
    nq, nk, d, dv = sum(lq) * case["heads"], sum(lk) * case["kv_heads"], case["dim"], case["dim_v"]
    if op == "differ":
        return {"bytes": size * (nq * (2 * d + 2 * dv) + nk * (2 * d + dv)) + 8 * nq,
                "flops": pairs * (4 * d + 2 * dv)}
    return {"bytes": size * (nq * (4 * d + 3 * dv) + 2 * nk * (2 * d + dv)) + 8 * nq,
            "flops": pairs * (12 * d + 4 * dv)}


# ------------------------------------------------------------------ inputs ---

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dtype = torch.float32 if case["dtype"] == F32 else torch.bfloat16

    def normal(*shape, mean=0.0):
        return (torch.randn(*shape, generator=gen, device=dev) + mean).to(dtype)

    def offsets(lens):
        at = [0]
        for n in lens:
            at.append(at[-1] + n)
        return torch.tensor(at, dtype=torch.int32, device=dev)

    def mask(n):
        """About one node in ten is padding."""
        if not case["masked"]:
            return None
        return (torch.rand(n, generator=gen, device=dev) >= 0.1).to(torch.uint8)

    s = {"op": case["op"]}
    if case["op"].startswith("turn"):
        n, h, d, pairs, axes = (case[t] for t in ("rows", "heads", "dim", "pairs", "axes"))
        # the projection that holds the rotated heads may hold the values too
        x = normal(n, h + 2 if case["packed"] else h, d)[:, :h]
        # wave lengths from 2 pi to a hundred times that, along the axes in turn or in any direction
        size = 0.01 ** (torch.arange(pairs, device=dev).float() / max(pairs, 2))
        if case["mixed"]:
            way = torch.randn(pairs, axes, generator=gen, device=dev)
            way = way / way.norm(dim=1, keepdim=True)
        else:
            way = torch.eye(axes, device=dev)[torch.arange(pairs, device=dev) % axes]
        s.update(x=x, waves=(way * size[:, None]).contiguous(), layout=case["layout"], mask=mask(n),
                 positions=case["box"] * torch.rand(n, axes, generator=gen, device=dev))
        if case["op"] == "turn_grad":
            # gradients follow the features in part, so the angles' gradients do not average out
            swap = torch.cat([x[..., 1:], x[..., :1]], 2)
            s["grad"] = (normal(n, h, d).float() + 0.5 * swap.float()).to(dtype)
        return s
    if case["op"].startswith("rms"):
        n, c = case["rows"], case["channels"]
        # a block of features with other components beside it in each row: strided rows
        x = (1.5 * normal(n, c + case["spare"]))[:, :c]
        s.update(x=x, groups=case["groups"], mask=mask(n), residual=normal(n, c) if case["residual"] else None,
                 weight=1 + 0.2 * torch.randn(case["period"], generator=gen, device=dev))
        if case["op"] == "rms_grad":
            s["grad"] = (normal(n, c).float() + 0.3 * x.float()).to(dtype)
            s["grad_total"] = s["residual"]
            s["residual"] = None
            s["rstd"] = _plain_rms(s)[2]
        return s
    lq, lk = _lengths_of(case)
    nq, nk, h, hk, d, dv = sum(lq), sum(lk), case["heads"], case["kv_heads"], case["dim"], case["dim_v"]
    if lq is lk:                                # one projection's output holds the maps' queries and keys
        rows = normal(nq, 2 * h + 2 * hk, d)
        s.update(q=rows[:, :2 * h], k=rows[:, 2 * h:])
    else:
        s.update(q=normal(nq, 2 * h, d), k=normal(nk, 2 * hk, d))
    s.update(v=normal(nk, hk, dv, mean=0.5), lam=0.2 + 0.6 * torch.rand(h, generator=gen, device=dev),
             q_ptr=offsets(lq), longest_q=max(lq), longest_k=max(lk), scale=1.0 / math.sqrt(d))
    s["k_ptr"] = s["q_ptr"] if lq is lk else offsets(lk)
    s["k_mask"] = mask(nk)
    s["q_mask"] = s["k_mask"] if lq is lk else None
    if case["op"] == "differ_grad":
        s["out"], s["second"], s["lse"] = _plain_differ(s)
        s["grad"] = normal(nq, h, dv, mean=0.3)
    return s


# ------------------------------------------------------------- plain forms ---

def _pairs_of(t, pairs, layout):
    """First and second elements of the rotated pairs, and the elements beyond them."""
    if layout == "halves":
        return t[..., :pairs], t[..., pairs:2 * pairs], t[..., 2 * pairs:]
    return t[..., 0:2 * pairs:2], t[..., 1:2 * pairs:2], t[..., 2 * pairs:]


def _joined(u, v, rest, layout):
    both = [u, v] if layout == "halves" else [torch.stack([u, v], -1).flatten(-2)]
    return torch.cat(both + [rest], -1)


def _turned(s, t, sign, wide=torch.float32):
    """The rows of t turned by sign times their angles; zeros in place of masked rows."""
    angle = s["positions"].double() @ s["waves"].double().T
    c, w = torch.cos(angle).to(wide)[:, None], (sign * torch.sin(angle)).to(wide)[:, None]
    u, v, rest = _pairs_of(_kept(s, t.to(wide)), s["waves"].shape[0], s["layout"])
    return u * c - v * w, u * w + v * c, rest


def _kept(s, t):
    """Zeros in place of masked rows."""
    return t if s["mask"] is None else torch.where((s["mask"] != 0).view(-1, *[1] * (t.dim() - 1)), t, 0.0)


def _plain_turn(s):
    return _joined(*_turned(s, s["x"], 1.0), s["layout"]).to(s["x"].dtype)


def _plain_turn_grad(s):
    gu, gv, rest = _turned(s, s["grad"], -1.0)
    u, v, _ = _pairs_of(_kept(s, s["x"].float()), gu.shape[-1], s["layout"])
    d_angle = (u * gv - v * gu).sum(1)
    d_positions = d_angle @ s["waves"]
    d_waves = (d_angle.double().T @ _kept(s, s["positions"]).double()).float()
    return _joined(gu, gv, rest, s["layout"]).to(s["x"].dtype), d_positions, d_waves


def _rms_parts(s, total):
    """Rows as (row, group, channel), and rstd."""
    parts = total.reshape(total.shape[0], s["groups"], -1)
    return parts, 1 / torch.sqrt((parts * parts).mean(2) + EPS)


def _weights(s, channels):
    return s["weight"].repeat(channels // s["weight"].numel()).reshape(s["groups"], -1)


def _plain_rms(s):
    x = s["x"]
    total = _kept(s, x.float() if s["residual"] is None else x.float() + s["residual"].float())
    parts, rstd = _rms_parts(s, total)
    y = parts * rstd[..., None] * _weights(s, x.shape[1])
    return y.reshape(x.shape).to(x.dtype), total.to(x.dtype) if s["residual"] is not None else None, rstd


def _plain_rms_grad(s):
    x = s["x"]
    parts, rstd = _kept(s, x.float()).reshape(x.shape[0], s["groups"], -1), s["rstd"][..., None]
    g, xh = _kept(s, s["grad"].float()).reshape(parts.shape), parts * rstd
    dn = g * _weights(s, x.shape[1])
    dx = (dn - xh * (dn * xh).mean(2, keepdim=True)) * rstd
    dx = dx.reshape(x.shape)
    if s["grad_total"] is not None:
        dx = _kept(s, dx + s["grad_total"].float())
    return dx.to(x.dtype), (g * xh).sum(0).reshape(-1, s["weight"].numel()).sum(0)


def _padded(ptr, longest):
    """(graph, position) -> row, and which of these are rows of the graph."""
    at = ptr[:-1, None].long() + torch.arange(longest, device=ptr.device)
    ok = at < ptr[1:, None]
    return torch.where(ok, at, 0), ok


def _rows(ptr, n):
    """Row -> graph and position in it."""
    r = torch.arange(n, device=ptr.device)
    g = torch.searchsorted(ptr[1:], r.to(torch.int32), right=True)
    return g, r - ptr[g]


def _differ_parts(s):
    """Padded (graph, key head, rows, dim) operands in fp32 and both maps' probabilities."""
    q, k, v = s["q"], s["k"], s["v"]
    iq, okq = _padded(s["q_ptr"], s["longest_q"])
    ik, okk = _padded(s["k_ptr"], s["longest_k"])
    if s["q_mask"] is not None:
        okq = okq & (s["q_mask"][iq] != 0)
    if s["k_mask"] is not None:
        okk = okk & (s["k_mask"][ik] != 0)
    b, lq = iq.shape
    hk, group = v.shape[1], q.shape[1] // k.shape[1]

    def heads(t, i, ok, g):
        t = torch.where(ok[:, :, None, None], t.float()[i], 0.0)          # (b, l, heads, d)
        t = t.reshape(b, i.shape[1], hk, g, t.shape[-1]).permute(0, 2, 1, 3, 4)
        return t.reshape(b, hk, i.shape[1] * g, t.shape[-1])

    row_ok = okq[:, None, :, None].expand(b, hk, lq, group).reshape(b, hk, lq * group)

    def softmax(qf, kf):
        sc = torch.matmul(qf, kf.transpose(2, 3)).mul_(s["scale"])
        sc.masked_fill_(~okk[:, None, None, :], -math.inf)
        top = sc.amax(3, keepdim=True)
        top = torch.where(torch.isfinite(top), top, 0.0)
        p = sc.sub_(top).exp_()
        p.masked_fill_(~row_ok[..., None], 0.0)
        total = p.sum(3, keepdim=True)
        lse = top + total.log()
        return p.div_(torch.where(total > 0, total, 1.0)), lse

    qf = [heads(q[:, m::2], iq, okq, group) for m in (0, 1)]
    kf = [heads(k[:, m::2], ik, okk, 1) for m in (0, 1)]
    maps = [softmax(*t) for t in zip(qf, kf)]
    return qf, kf, heads(v, ik, okk, 1), [p for p, _ in maps], [t for _, t in maps], (iq, okq), heads


def _to_rows(t, ptr, n, group):
    """(graph, key head, position x group, dim) back to (row, head, dim)."""
    b, hk, r, d = t.shape
    g, pos = _rows(ptr, n)
    t = t.reshape(b, hk, r // group, group, d).permute(0, 2, 1, 3, 4)
    return t.reshape(b, r // group, hk * group, d)[g, pos]


def _lam_of_rows(s, hk, rows):
    """lam of each (key head, position x group)."""
    return s["lam"].reshape(hk, 1, -1).expand(hk, rows // (s["lam"].numel() // hk), -1).reshape(1, hk, rows, 1)


def _plain_differ(s):
    q, n = s["q"], s["q"].shape[0]
    group = q.shape[1] // s["k"].shape[1]
    _, _, vf, p, lse, _, _ = _differ_parts(s)
    first, second = (torch.matmul(t, vf) for t in p)
    out = first - _lam_of_rows(s, vf.shape[1], first.shape[2]) * second
    rows = lambda t: _to_rows(t, s["q_ptr"], n, group)
    return rows(out).to(q.dtype), rows(second).to(q.dtype), rows(torch.cat(lse, 3)).contiguous()


def _plain_differ_grad(s):
    q, k = s["q"], s["k"]
    group = q.shape[1] // k.shape[1]
    qf, kf, vf, p, _, (iq, okq), heads = _differ_parts(s)
    g = heads(s["grad"], iq, okq, group)
    lam = _lam_of_rows(s, vf.shape[1], g.shape[2])
    dv = torch.matmul((p[0] - lam * p[1]).transpose(2, 3), g)
    dp = torch.matmul(g, vf.transpose(2, 3))
    delta = [(t * dp).sum(3, keepdim=True) for t in p]
    d_lam = -_to_rows(delta[1], s["q_ptr"], q.shape[0], group).double().sum((0, 2)).float()
    dq, dk = [], []
    for m, factor in ((0, s["scale"]), (1, -lam * s["scale"])):
        ds = p[m].mul_(dp - delta[m]).mul_(factor)
        dq.append(_to_rows(torch.matmul(ds, kf[m]), s["q_ptr"], q.shape[0], group))
        dk.append(_to_rows(torch.matmul(ds.transpose(2, 3), qf[m]), s["k_ptr"], k.shape[0], 1))
    return (torch.stack(dq, 2).flatten(1, 2).to(q.dtype), torch.stack(dk, 2).flatten(1, 2).to(q.dtype),
            _to_rows(dv, s["k_ptr"], k.shape[0], 1).to(q.dtype), d_lam)


def run(state):
    s = state
    if not own:
        return {"turn": _plain_turn, "turn_grad": _plain_turn_grad, "differ": _plain_differ,
                "differ_grad": _plain_differ_grad, "rms": _plain_rms, "rms_grad": _plain_rms_grad}[s["op"]](s)
    from equivariant_gnn_message_amd import e3conv as E
    if s["op"] == "turn":
        return E.e3conv_rotary(s["x"], s["positions"], s["waves"], s["layout"], row_mask=s["mask"])
    if s["op"] == "turn_grad":
        return E.e3conv_rotary_backward(s["x"], s["positions"], s["waves"], s["grad"], s["layout"],
                                        row_mask=s["mask"])
    if s["op"] == "differ":
        return E.e3conv_diff_attention(s["q"], s["k"], s["v"], s["lam"], s["q_ptr"], s["k_ptr"], s["scale"],
                                       q_mask=s["q_mask"], k_mask=s["k_mask"])
    if s["op"] == "differ_grad":
        return E.e3conv_diff_attention_backward(s["q"], s["k"], s["v"], s["lam"], s["out"], s["second"], s["lse"],
                                                s["grad"], s["q_ptr"], s["k_ptr"], s["scale"], q_mask=s["q_mask"],
                                                k_mask=s["k_mask"])
    if s["op"] == "rms":
        return E.e3conv_rms_norm(s["x"], s["weight"], s["groups"], EPS, residual=s["residual"], row_mask=s["mask"])
    return E.e3conv_rms_norm_backward(s["x"], s["weight"], s["groups"], s["rstd"], s["grad"],
                                      grad_total=s["grad_total"], row_mask=s["mask"])


# ------------------------------------------------------------ 64-bit values ---

def exact(case, seed):
    """The operators' definition in 64 bits: rotations as complex products, attention graph by graph, the
    norm's gradient by differentiation."""
    s = prepare(case, seed)
    if case["op"].startswith("turn"):
        return _exact_turn(case, s)
    return _exact_rms(case, s) if case["op"].startswith("rms") else _exact_differ(case, s)


def _exact_turn(case, s):
    n, p = case["pairs"], s["positions"].double()
    first = torch.arange(n, device=p.device) * (1 if case["layout"] == "halves" else 2)
    second = first + (n if case["layout"] == "halves" else 1)
    dead = None if s["mask"] is None else s["mask"] == 0

    def wide(t):
        t = t.double()
        if dead is not None:
            t[dead] = 0
        return t

    angle = (p[:, None, :] * s["waves"].double()).sum(2)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    x = wide(s["x"])
    if "grad" not in s:
        z = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        return x
    g = wide(s["grad"])
    z = torch.complex(g[..., first], g[..., second]) * turn.conj()
    d_angle = (torch.complex(x[..., first], x[..., second]).conj() * z).imag.sum(1)
    g[..., first], g[..., second] = z.real, z.imag
    return g, (d_angle[:, :, None] * s["waves"].double()).sum(1), torch.matmul(d_angle.T, p)


def _exact_rms(case, s):
    x = s["x"].double()
    live = torch.ones(x.shape[0], 1, dtype=torch.bool, device=x.device) if s["mask"] is None else (s["mask"] != 0)[:, None]
    w = s["weight"].double().requires_grad_("grad" in s)
    if "grad" in s:
        x = torch.where(live, x, 0.0).requires_grad_()
    with torch.enable_grad():
        total = torch.where(live, x if s["residual"] is None else x + s["residual"].double(), 0.0)
        rows = total.unflatten(1, (case["groups"], -1))
        rstd = (rows.square().mean(2) + EPS).rsqrt()
        y = (rows * rstd[..., None]).flatten(1) * w.tile(case["channels"] // case["period"])
        if "grad" not in s:
            return y, total if s["residual"] is not None else None, rstd
        dx, dw = torch.autograd.grad(y, (x, w), torch.where(live, s["grad"].double(), 0.0))
    if s["grad_total"] is not None:
        dx = dx + s["grad_total"].double()
    return torch.where(live, dx, 0.0), dw


def _exact_differ(case, s):
    lq, lk = _lengths_of(case)
    q, k, v, lam = (s[t].double() for t in ("q", "k", "v", "lam"))
    group = q.shape[1] // k.shape[1]
    grad = s["grad"].double() if "grad" in s else None
    n, h = q.shape[0], lam.numel()
    out, second = (q.new_zeros(n, h, v.shape[2]) for _ in range(2))
    lse = q.new_full((n, h, 2), -math.inf)
    dq, dk, dv, d_lam = (torch.zeros_like(t) for t in (q, k, v, lam))
    a = b = 0
    for nq, nk in zip(lq, lk):
        rows, cols = torch.arange(a, a + nq, device=q.device), torch.arange(b, b + nk, device=q.device)
        a, b = a + nq, b + nk
        if s["q_mask"] is not None:
            rows = rows[s["q_mask"][rows] != 0]
        if s["k_mask"] is not None:
            cols = cols[s["k_mask"][cols] != 0]
        if not len(rows) or not len(cols):
            continue
        for i in range(h):
            j = i // group
            p = []
            for m in (0, 1):
                logits = (q[rows, 2 * i + m] @ k[cols, 2 * j + m].T) * s["scale"]
                lse[rows, i, m] = torch.logsumexp(logits, 1)
                p.append(torch.exp(logits - lse[rows, i, m][:, None]))
                del logits
            if grad is None:
                second[rows, i] = p[1] @ v[cols, j]
                out[rows, i] = p[0] @ v[cols, j] - lam[i] * second[rows, i]
                continue
            g = grad[rows, i]
            dp = g @ v[cols, j].T
            dv[cols, j] += (p[0] - lam[i] * p[1]).T @ g
            d_lam[i] -= (p[1] * dp).sum()
            for m in (0, 1):
                d = p[m] * dp
                ds = (d - p[m] * d.sum(1, keepdim=True)) * (s["scale"] if m == 0 else -s["scale"] * lam[i])
                dq[rows, 2 * i + m] = ds @ k[cols, 2 * j + m]
                dk[cols, 2 * j + m] += ds.T @ q[rows, 2 * i + m]
                del d, ds
            del dp, p
    return (out, second, lse) if grad is None else (dq, dk, dv, d_lam)
