"""Where differential attention reads and writes: memory beside its results, and rows at the ends of what a tile's 32-bit
offsets reach."""

import numpy as np
import pytest

from equivariant_gnn_message_amd import e3conv as E

from ._gpu import say
from .test_gpu_attention import dev, ptr
from .test_gpu_diff_attention import draw

pytestmark = pytest.mark.gpu

GUARD = 7.0


class Guarded:
    """Tensors inside larger storage of guard values, and whether those are as they were."""

    def __init__(self):
        self.held = []

    def rows(self, like):
        """As `like` (rows, heads, dim), with rows before and after it, one head and one element more."""
        import torch
        n, h, d = like.shape
        store = torch.full((n + 4, h + 1, d + 8), GUARD, dtype=like.dtype, device="cuda")
        inner = torch.zeros(store.shape, dtype=torch.bool, device="cuda")
        inner[2:n + 2, :h, :d] = True
        self.held.append((store, inner))
        return store[2:n + 2, :h, :d]

    def flat(self, n, dtype):
        import torch
        store = torch.full((n + 128,), GUARD, device="cuda").to(dtype)
        inner = torch.zeros(store.shape, dtype=torch.bool, device="cuda")
        inner[64:64 + n] = True
        self.held.append((store, inner))
        return store[64:64 + n]

    def intact(self):
        return all(bool((store[~inner] == GUARD).all()) for store, inner in self.held)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,dv", [(32, 64), (64, 128), (20, 33)])
@pytest.mark.parametrize("n", [3, 200, 3000])
def test_nothing_beside_the_results_is_written(dtype, d, dv, n):
    """Offsets that decrease, start past 0, are negative or leave the tensors, and such as they should be: results,
    gradients, statistics and workspaces inside guard values, which stay."""
    import torch
    q, k, v, lam, g = draw(55, dtype, [n], [n], 2, 1, d, dv)
    args = lambda p: E._diff_attention_args(q, k, v, lam, p, p, None, None, None)[0]
    for offsets in ([0, n], [0, n // 2, n // 2, n], [5, 150, 60, 200], [-7, 90, 400, 200], [0, n, n, n // 2],
                    [n, 0, 0, n], [2 ** 30, -2 ** 31, 2 ** 31 - 1, 0]):
        p = dev(np.array(offsets, np.int32))
        say(f"[diff] {dtype} {d} {dv} {n} nodes, offsets {offsets}")
        in_, held = E.e3conv_diff_attention_workspace_size, Guarded()
        out, second = held.rows(g), held.rows(g)
        lse = held.flat(2 * n * 2, torch.float32)
        E.e3conv_diff_attention(q, k, v, lam, p, p, out=out, second=second, lse=lse,
                                workspace=held.flat(in_(args(p)), torch.uint8))
        grads = [held.rows(t) for t in (q, k, v)]
        E.e3conv_diff_attention_backward(q, k, v, lam, out, second, lse, g, p, p, grads=grads,
                                         workspace=held.flat(in_(args(p), True), torch.uint8))
        torch.cuda.synchronize()
        assert held.intact(), offsets


@pytest.mark.parametrize("heads,d,dv", [((1, 1), 64, 128), ((1, 1), 32, 64), ((2, 1), 64, 128)])
@pytest.mark.parametrize("step", [(1 << 25) - (1 << 12), 1 << 25])
def test_rows_at_the_reach_of_32_bit_offsets(heads, d, dv, step):
    """Tiles of rows that span just less than 4 GiB (offsets of 32 bits, past 2^31 too) and just as much (64 bits), for
    every operand and result: the dense call's bits."""
    import torch
    n = 70
    q, k, v, lam, g = draw(61, "bf16", [n], [n], *heads, d, dv)
    p = dev(ptr([n]))
    ref = E.e3conv_diff_attention(q, k, v, lam, p, p)
    want = E.e3conv_diff_attention_backward(q, k, v, lam, *ref, g, p, p)
    store = torch.empty(n * step, dtype=torch.bfloat16, device="cuda").view(n, step)
    at = 0

    def far(t, fill=True):
        nonlocal at
        width = t.shape[1] * t.shape[2]
        view = store[:, at:at + width].unflatten(1, t.shape[1:])
        at += width
        return view.copy_(t) if fill else view

    say(f"[diff] rows {step} apart, heads {heads} {d} {dv}")
    fq, fk, fv, fg = map(far, (q, k, v, g))
    out, second = far(ref[0], False), far(ref[1], False)
    lse = E.e3conv_diff_attention(fq, fk, fv, lam, p, p, out=out, second=second)[2]
    grads = [far(t, False) for t in (q, k, v)]
    glam = E.e3conv_diff_attention_backward(fq, fk, fv, lam, out, second, lse, fg, p, p, grads=grads)[3]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((out, second, lse), ref))
    assert all(torch.equal(a, b) for a, b in zip((*grads, glam), want))
