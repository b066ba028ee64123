"""Attention and group norm on a stream that is not the current one: what a call allocates is not memory
that work still queued on the current stream reads."""

import pytest

from equivariant_gnn_message_amd import e3conv as E

from .test_gpu_attention import dev, ptr

pytestmark = pytest.mark.gpu

ROWS, HEADS, DIM = 8192, 4, 64          # rows x heads x dim fp32: 8 MiB


def calls():
    """name -> call(stream) with 8 MiB results, its operands ready on every stream."""
    import torch
    gen = torch.Generator().manual_seed(1)
    q, k, v, g = (torch.randn((ROWS, HEADS, DIM), generator=gen).cuda() for _ in range(4))
    lens = [64] * (ROWS // 64)
    p = dev(ptr(lens))
    out, lse = E.e3conv_attention(q, k, v, p, p)
    x, gy = q.view(ROWS, -1), g.view(ROWS, -1)
    w = torch.ones(HEADS * DIM, device="cuda")
    _, mean, rstd = E.e3conv_group_norm(x, p, 8, w, w, activation="silu")
    torch.cuda.synchronize()
    return {
        "attention": lambda s: E.e3conv_attention(q, k, v, p, p, stream=s),
        "attention backward": lambda s: E.e3conv_attention_backward(q, k, v, out, lse, g, p, p, stream=s),
        "group norm": lambda s: E.e3conv_group_norm(x, p, 8, w, w, activation="silu", stream=s),
        "group norm backward": lambda s: E.e3conv_group_norm_backward(x, p, 8, w, w, "silu", mean, rstd, gy, stream=s),
    }


@pytest.mark.parametrize("name", ["attention", "attention backward", "group norm", "group norm backward"])
@pytest.mark.parametrize("handle", [False, True])
def test_memory_still_read_on_the_current_stream(name, handle):
    """Freed tensors of the results' size, read by copies behind queued products, keep their values."""
    import torch
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    a = torch.ones((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    freed = [torch.full((ROWS, HEADS, DIM), float(i), device="cuda") for i in range(6)]
    held = {t.data_ptr() for t in freed}
    kept = [torch.empty_like(t) for t in freed]
    for _ in range(20):
        a = a @ a * 2.0 ** -12                # some milliseconds of work before the copies
    for to, t in zip(kept, freed):
        to.copy_(t)
    del freed, t
    got = call(side.cuda_stream if handle else side)
    assert not held & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    for i, t in enumerate(kept):
        assert bool((t == i).all()), i
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_default_stream_from_a_side_stream():
    import torch
    call = calls()["attention"]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    for stream in (torch.cuda.default_stream(), 0):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = call(stream)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
