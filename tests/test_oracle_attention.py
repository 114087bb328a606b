"""The oracle of head norms and attention (CPU): closed forms, invariants, differences."""

import numpy as np
import pytest

from oracle import attention as A
from oracle import heads as H

RNG = np.random.default_rng


def _tables(P, pairs, seed=0):
    a = RNG(seed).uniform(-3, 3, (P, pairs))
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("layout", ["pairs", "halves"])
def test_a_rotation_keeps_lengths_and_adds_angles(layout):
    x = RNG(1).normal(size=(5, 2, 8))
    a = np.arange(20)[:, None] * np.array([1.0, 0.3, 0.01])
    cos, sin = np.cos(a), np.sin(a)
    y = H.forward(x, "none", None, cos, sin, np.full(5, 4), layout)
    np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    np.testing.assert_array_equal(y[..., 6:], x[..., 6:])   # past the three pairs
    again = H.forward(y, "none", None, cos, sin, np.full(5, 7), layout)
    np.testing.assert_allclose(again, H.forward(x, "none", None, cos, sin, np.full(5, 11), layout))
    # position 0 turns nothing
    np.testing.assert_array_equal(H.forward(x, "none", None, cos, sin, np.zeros(5, int), layout), x)


def test_rotated_scores_depend_on_the_distance_alone():
    a = np.arange(30)[:, None] * np.array([1.0, 0.2])
    q, k = RNG(2).normal(size=(2, 1, 1, 4))
    def dot(i, j):
        return float((H.forward(q, "none", None, np.cos(a), np.sin(a), [i])
                      * H.forward(k, "none", None, np.cos(a), np.sin(a), [j])).sum())
    assert abs(dot(3, 8) - dot(20, 25)) < 1e-12


@pytest.mark.parametrize("norm", ["rms", "layer", "none"])
@pytest.mark.parametrize("layout", ["pairs", "halves"])
def test_head_gradients_are_differences(norm, layout):
    r = RNG(3)
    x, dy, w = r.normal(size=(4, 3, 10)) + 0.2, r.normal(size=(4, 3, 10)), r.normal(size=10)
    cos, sin = _tables(6, 3)
    kw = dict(norm=norm, cos=cos, sin=sin, positions=[2, -1, 5, 6], layout=layout)
    w = None if norm == "none" else w
    dx, dw = H.backward(dy, x, w=w, **kw)
    f = lambda x, w: (H.forward(x, w=w, **kw) * dy).sum()
    h = 1e-5
    for at in [(0, 0, 0), (0, 2, 9), (2, 1, 4), (1, 0, 3), (3, 2, 1)]:
        e = np.zeros_like(x)
        e[at] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    assert not dx[1].any() and not dx[3].any()
    if w is not None:
        for i in range(10):
            e = np.zeros(10)
            e[i] = h
            assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_attention_of_one_key_is_its_value():
    r = RNG(4)
    q, k, v = r.normal(size=(3, 2, 8)), r.normal(size=(1, 1, 8)), r.normal(size=(1, 1, 8))
    o, lse = A.forward(q, k, v, A.allowed(3, 1), 0.3)
    np.testing.assert_allclose(o, np.broadcast_to(v, o.shape))
    np.testing.assert_allclose(lse, 0.3 * (q * k).sum(-1))


def test_equal_scores_give_the_mean_and_lengths_end_it():
    v = RNG(5).normal(size=(6, 1, 8))
    q, k = np.zeros((4, 1, 8)), np.zeros((6, 1, 8))
    ok = A.allowed(4, 6, [0, 1, 2, 3], [0, 3, 3, 6], [2, 0, 9], [1, 1, 1, 0, 1, 1])
    o, lse = A.forward(q, k, v, ok, 1.0)
    np.testing.assert_allclose(o[0, 0], v[:2, 0].mean(0))
    assert not o[1].any() and lse[1, 0] == -np.inf          # a sequence without keys
    np.testing.assert_allclose(o[2, 0], v[4:, 0].mean(0))   # a masked key
    assert not o[3].any() and lse[3, 0] == -np.inf          # of no sequence
    np.testing.assert_allclose(lse[[0, 2], 0], np.log(2))


def test_masked_elements_reach_nothing():
    r = RNG(6)
    q, k, v, do = (r.normal(size=(4, 2, 8)) for _ in range(4))
    ok = A.allowed(4, 4, key_mask=[1, 0, 1, 1])
    o, lse = A.forward(q, k, v, ok, 0.5)
    want = A.backward(do, q, k, v, o, lse, ok, 0.5)
    k[1], v[1] = np.nan, np.inf
    for a, b in zip(A.forward(q, k, v, ok, 0.5) + A.backward(do, q, k, v, o, lse, ok, 0.5), (o, lse) + want):
        np.testing.assert_array_equal(a, b)
    assert not want[1][1].any() and not want[2][1].any()


def test_attention_gradients_are_differences():
    r = RNG(7)
    q, k, v = r.normal(size=(5, 4, 8)), r.normal(size=(7, 2, 8)), r.normal(size=(7, 2, 8))
    do = r.normal(size=q.shape)
    ok = A.allowed(5, 7, [0, 2, 4], [0, 3, 7], None, [1, 1, 1, 1, 0, 1, 1])
    o, lse = A.forward(q, k, v, ok, 0.4)
    grads = A.backward(do, q, k, v, o, lse, ok, 0.4)
    h = 1e-5
    for n, (x, g) in enumerate(zip((q, k, v), grads)):
        for _ in range(8):
            at = tuple(r.integers(0, s) for s in x.shape)
            vals = []
            for sign in (h, -h):
                args = [q, k, v]
                args[n] = x.copy()
                args[n][at] += sign
                vals.append((A.forward(*args, ok, 0.4)[0] * do).sum())
            assert abs((vals[0] - vals[1]) / (2 * h) - g[at]) < 1e-7
