"""Pins for the oracle of the 8-bit layer and the gated norms (CPU only).

* codes against hand-worked values, every E4M3 value a fixed point, rounding off by
  at most half a step, the scale's definition by its two inequalities, power-of-two
  equivariance, square blocks that transpose;
* the layer's gradients and the norms' against central differences of the forward.
"""

import numpy as np
import pytest

from oracle import fp8, norm
from oracle.formats import E4M3_VALUES


def test_hand_worked_blocks():
    v = np.zeros((1, 256))
    v[0, :6] = [448.0, 17.0, 18.0, 19.0, -0.0009765625, 0.0029296875]   # S = 1
    v[0, 128:131] = [449.0, -2.0, np.inf]                               # S = 2
    c, s = fp8.quantize(v)
    assert s.tolist() == [[127, 128]]
    # 17 ties between 16 and 18: 16 (even code); 19 between 18 and 20: 20; -2^-10 and
    # 1.5 * 2^-9 tie between subnormals 0 | 2^-9 and 2^-9 | 2^-8: -0 and 2^-8
    assert E4M3_VALUES[c[0, :6]].tolist() == [448.0, 16.0, 18.0, 20.0, 0.0, 0.00390625]
    assert c[0, 4] == 0x80
    # 449 / 2 = 224.5 -> 224; -1; infinity -> NaN code
    assert E4M3_VALUES[c[0, 128]] == 224.0 and E4M3_VALUES[c[0, 129]] == -1.0
    assert c[0, 130] == 0x7F


def test_format_properties():
    rng = np.random.default_rng(0)
    v = rng.standard_normal((7, 300)) * np.exp2(rng.integers(-20, 20, (7, 1)))
    c, s = fp8.quantize(v)
    assert c.shape == (7, 384) and s.shape == (7, 3) and not c[:, 300:].any()
    p = np.zeros((7, 384))
    p[:, :300] = v
    top = np.abs(p).reshape(7, 3, 128).max(axis=2)
    S = np.exp2(s.astype(float) - 127)
    assert (top / S <= 448).all() and (top / (S / 2) > 448).all()
    q = fp8.values(c, s, 384)
    unit = S.repeat(128, axis=1)
    # half a step: 2^-4 of the value, or 2^-10 of the scale below the normals
    assert (np.abs(q - p) <= np.maximum(np.abs(p) / 16, unit / 1024)).all()
    c2, s2 = fp8.quantize(v * 64)
    assert np.array_equal(c, c2) and np.array_equal(s2, s + 6)
    w = rng.standard_normal((200, 300))
    assert np.array_equal(fp8.held(w, True), fp8.held(w.T, True).T)
    grid = np.zeros((1, 128))
    grid[0, :127] = E4M3_VALUES[:127]
    assert np.array_equal(fp8.held(grid), grid)


def test_layout_of_scales():
    b = np.arange(12, dtype=np.uint8).reshape(2, 6)
    want = [[[0, 1, 2, 3], [6, 7, 8, 9]], [[4, 5, 127, 127], [10, 11, 127, 127]]]
    assert fp8.layout_scales(b).tolist() == want


def test_layer_gradients_against_differences():
    # whole numbers that the format holds exactly, so that it is linear in them
    rng = np.random.default_rng(1)
    x, w, dy = (rng.integers(-4, 5, s).astype(float) for s in ((5, 40), (6, 40), (5, 6)))
    dx, dw, db = fp8.backward(dy, x, w)
    d = rng.integers(-2, 3, x.shape)
    assert ((fp8.forward(x + d, w) - fp8.forward(x, w)) * dy).sum() == (dx * d).sum()
    d = rng.integers(-2, 3, w.shape)
    assert ((fp8.forward(x, w + d) - fp8.forward(x, w)) * dy).sum() == (dw * d).sum()
    assert np.array_equal(db, dy.sum(axis=0))


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["rms", "layer"])
def test_norm_gradients_against_differences(post, pre):
    rng = np.random.default_rng(2)
    M, C, off = 7, 9, [0, 3, 3, 6]
    seq = norm.sequences(M, off)
    live = (seq >= 0)[:, None]
    inputs = {"x": rng.standard_normal((M, C)), "y": rng.standard_normal((M, C)),
              "gate": rng.standard_normal((3, C)), "weight": rng.standard_normal(C),
              "bias": rng.standard_normal(C), "scale": rng.standard_normal((3, C)),
              "shift": rng.standard_normal((3, C))}
    if post != "none":
        inputs["post_weight"] = rng.standard_normal(C)
    dh, dn = rng.standard_normal((M, C)), rng.standard_normal((M, C))

    def forward(i):
        h = norm.stream(i["x"], i["y"], seq, 0.7, post, i.get("post_weight"), i["gate"])
        n = norm.prenorm(h, seq, pre, i["weight"], i["bias"], i["scale"], i["shift"])
        return h, n

    def loss(i):
        h, n = forward(i)
        return ((h * dh + n * dn) * live).sum()

    h, _ = forward(inputs)
    g = norm.backward(dh, dn, h, inputs["y"], seq, 3, 0.7, post, inputs.get("post_weight"),
                      inputs["gate"], pre, inputs["weight"], inputs["bias"], inputs["scale"])
    for name, v in inputs.items():
        d = rng.standard_normal(v.shape)
        step = 1e-5
        up, down = ({**inputs, name: v + k * step * d} for k in (1, -1))
        diff = (loss(up) - loss(down)) / (2 * step)
        want = (g[{"x": "dx", "y": "dy"}.get(name, name)] * d).sum()
        # the difference is off by step^2 f'''/6 and by 2^-53 |f| / step: 1e-9 of O(10) terms
        assert abs(diff - want) <= 1e-7 * max(1.0, abs(want)), (name, diff, want)
