"""The float64 attention oracle: hand-worked rows, brute force over single rows,
and central differences for both gradients."""
import math

import numpy as np
import pytest

from oracle import attention as A

RNG = np.random.default_rng


def test_hand_worked_rotation_and_norm():
    table = A.rope_table(4, 2, base=100.0)
    assert table.shape == (4, 2) and table[0].tolist() == [1.0, 0.0]
    x = np.array([[[3.0, 4.0]]])                        # mean square 12.5
    z = A.norm_rope(x, np.array([2]), table, np.array([2.0, 1.0]), 0.0)
    a, b = 2 * 3 / math.sqrt(12.5), 4 / math.sqrt(12.5)
    c, s = float(table[2, 0]), float(table[2, 1])
    np.testing.assert_allclose(z[0, 0], [a * c - b * s, a * s + b * c], rtol=1e-12)


def test_pair_layouts_are_permutations_of_each_other():
    rng = RNG(1)
    table, pos = A.rope_table(9, 8), np.array([5, 8])
    x = rng.standard_normal((2, 3, 10))
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7, 8, 9])     # interleaved element -> its place in halves
    z = A.rotate(x, pos, table, True)
    np.testing.assert_allclose(A.rotate(x[..., order], pos, table, False), z[..., order], rtol=1e-12)
    np.testing.assert_allclose(A.rotate(z, pos, table, True, back=True), x, rtol=1e-6, atol=1e-6)


def test_visibility():
    assert A.visible(3, 3).tolist() == [[True, False, False], [True, True, False], [True, True, True]]
    assert A.visible(1, 5, window=2, sinks=1).tolist() == [[True, False, False, True, True]]
    assert A.visible(3, 2).tolist() == [[False, False], [True, False], [True, True]]


@pytest.mark.parametrize("nq,nk,window,sinks", [(5, 5, 0, 0), (4, 9, 3, 2), (6, 4, 0, 0), (1, 7, 1, 0)])
def test_attention_against_single_rows(nq, nk, window, sinks):
    rng = RNG(nq * 10 + nk)
    q, k, v = rng.standard_normal((nq, 4, 8)), rng.standard_normal((nk, 2, 8)), rng.standard_normal((nk, 2, 8))
    out, lse, _ = A.attention(q, k, v, window, sinks)
    for i in range(nq):
        p = i + nk - nq
        keys = [j for j in range(nk) if j <= p and (not window or j > p - window or j < sinks)]
        for h in range(4):
            if not keys:
                assert lse[h, i] == -np.inf and not out[i, h].any()
                continue
            w = [math.exp(sum(q[i, h, d] * k[j, h // 2, d] for d in range(8)) / math.sqrt(8)) for j in keys]
            assert lse[h, i] == pytest.approx(math.log(sum(w)), abs=1e-12)
            np.testing.assert_allclose(out[i, h], sum(x * v[j, h // 2] for x, j in zip(w, keys)) / sum(w), atol=1e-12)


def differences(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        y = x.copy()
        y[i] += h
        up = f(y)
        y[i] -= 2 * h
        g[i] = (up - f(y)) / (2 * h)
    return g


@pytest.mark.parametrize("window,sinks,nk", [(0, 0, 4), (2, 1, 6), (0, 0, 3)])
def test_attention_gradient_by_differences(window, sinks, nk):
    rng = RNG(7)
    q, k, v = rng.standard_normal((4, 2, 4)), rng.standard_normal((nk, 1, 4)), rng.standard_normal((nk, 1, 4))
    w = rng.standard_normal((4, 2, 4))
    out, lse, _ = A.attention(q, k, v, window, sinks)
    got = A.attention_backward(w, q, k, v, out, lse, window, sinks)
    args = [q, k, v]
    for n in range(3):
        def f(x, n=n):
            a = list(args)
            a[n] = x
            return float((A.attention(*a, window, sinks)[0] * w).sum())
        np.testing.assert_allclose(got[n], differences(f, args[n]), atol=1e-8)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_gradient_by_differences(interleaved):
    rng = RNG(3)
    x, g, w = rng.standard_normal((3, 2, 8)), rng.standard_normal(8), rng.standard_normal((3, 2, 8))
    table, pos = A.rope_table(50, 4), np.array([0, 7, 49])
    dx, dg = A.norm_rope_backward(w, x, pos, table, g, 1e-3, interleaved)
    f = lambda x, g: float((A.norm_rope(x, pos, table, g, 1e-3, interleaved) * w).sum())  # noqa: E731
    np.testing.assert_allclose(dx, differences(lambda y: f(y, g), x), atol=1e-7)
    np.testing.assert_allclose(dg, differences(lambda y: f(x, y), g), atol=1e-7)


def test_paged_rows():
    cache = np.arange(3 * 2 * 4 * 1).reshape(3, 2, 4, 1)
    rows = A.paged_rows(cache, [2, 0], 5)
    assert rows.shape == (5, 2, 1) and rows[:, 0, 0].tolist() == [16, 17, 18, 19, 0]
    assert A.paged_rows(cache, [0], 0).shape == (0, 2, 1)
