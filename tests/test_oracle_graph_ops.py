"""The attention and group-norm oracles against differences and closed forms (CPU)."""

import numpy as np
import pytest

from oracle import attention, norm


def _central(f, t, h=1e-5):
    d = np.zeros_like(t)
    for i in np.ndindex(*t.shape):
        keep = t[i]
        t[i] = keep + h
        up = f()
        t[i] = keep - h
        down = f()
        t[i] = keep
        d[i] = (up - down) / (2 * h)
    return d


def test_attention_gradients_equal_differences():
    rng = np.random.default_rng(0)
    q_ptr, k_ptr = [0, 3, 3, 5], [0, 4, 6, 6]     # the middle graph has no query, the last no key
    q, k, v = rng.standard_normal((5, 4, 3)), rng.standard_normal((6, 2, 3)), rng.standard_normal((6, 2, 2))
    g, k_mask = rng.standard_normal((5, 4, 2)), np.array([1, 0, 1, 1, 1, 1])
    run = lambda: attention.attention(q, k, v, q_ptr, k_ptr, 0.7, None, k_mask, g)
    res = run()
    f = lambda: float((run()["out"] * g).sum())
    for t, name in ((q, "dq"), (k, "dk"), (v, "dv")):
        np.testing.assert_allclose(res[name], _central(f, t), atol=2e-9, rtol=2e-7)
    assert np.all(res["out"][3:] == 0) and np.all(np.isneginf(res["lse"][3:]))
    assert np.all(res["dk"][1] == 0) and np.all(res["dv"][1] == 0)


def test_attention_closed_forms():
    """One key: out is its value; equal logits: the mean of the values, lse = log n + logit."""
    rng = np.random.default_rng(1)
    v = rng.standard_normal((3, 1, 4))
    q, k = np.ones((2, 1, 2)), np.ones((3, 1, 2))
    res = attention.attention(q, k, v, [0, 1, 2], [0, 1, 3], 0.5)
    np.testing.assert_allclose(res["out"][0], v[0])
    np.testing.assert_allclose(res["out"][1], v[1:].mean(0))
    np.testing.assert_allclose(res["lse"][:, 0], [1.0, 1.0 + np.log(2)])


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_group_norm_gradients_equal_differences(act):
    rng = np.random.default_rng(2)
    ptr, mask = [0, 4, 4, 5, 9], np.array([1, 1, 0, 1, 1, 1, 1, 1, 1])
    x, w, c = rng.standard_normal((9, 6)), rng.standard_normal(6), rng.standard_normal(6)
    g = rng.standard_normal((9, 6))
    run = lambda: norm.group_norm(x, ptr, 3, w, c, 1e-3, act, mask, g)[0]
    res = run()
    f = lambda: float((run()["y"] * g).sum())
    for t, name in ((x, "dx"), (w, "dw"), (c, "dc")):
        np.testing.assert_allclose(res[name], _central(f, t), atol=1e-7, rtol=1e-5)
    assert np.all(res["y"][2] == 0) and np.all(res["dx"][2] == 0)


def test_group_norm_statistics():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((50, 8)) * 3 + 7
    val, _ = norm.group_norm(x, [0, 20, 50], 2, None, None, 1e-12, "none")
    for a, b in ((0, 20), (20, 50)):
        y = val["y"][a:b].reshape(b - a, 2, 4)
        np.testing.assert_allclose(y.mean((0, 2)), 0, atol=1e-12)
        np.testing.assert_allclose((y ** 2).mean((0, 2)), 1, rtol=1e-9)
