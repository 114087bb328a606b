"""The gated norms around a transformer block in float64, forward and backward.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

    h = alpha x + gate[g] * post(y)
    n = (pre(h) w + b) (1 + scale[g]) + shift[g]

norm(v) = v / sqrt(mean(v^2) + eps) over the row ('rms'), or the same of
v - mean(v) ('layer'); post is times post_w, and 'none' leaves y.  ``seq`` maps a
row to its table row, -1 for rows of no sequence, which have no result.
"""

import numpy as np


def normed(v, kind, eps):
    """(the normed rows, 1 / their deviation)"""
    if kind == "layer":
        v = v - v.mean(axis=1, keepdims=True)
    r = 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)
    return v * r, r


def _back(g, v, r, kind):
    """Gradient through a norm with result v: r (g - v mean(g v)), less mean g for 'layer'."""
    d = g - v * (g * v).mean(axis=1, keepdims=True)
    return r * (d if kind == "rms" else d - g.mean(axis=1, keepdims=True))


def sequences(M, offsets):
    seq = np.full(M, -1) if offsets is not None else np.zeros(M, int)
    if offsets is not None:
        for g in range(len(offsets) - 1):
            seq[offsets[g]:offsets[g + 1]] = g
    return seq


def _rows(table, seq):
    return 0.0 if table is None else np.asarray(table, np.float64).reshape(-1, table.shape[-1])[seq]


def stream(x, y, seq, alpha=1.0, post="none", post_w=None, gate=None, eps=1e-6):
    """h"""
    if y is None:
        return alpha * x
    p = y if post == "none" else normed(y, post, eps)[0] * (1.0 if post_w is None else post_w)
    return alpha * x + (p if gate is None else _rows(gate, seq) * p)


def prenorm(h, seq, pre, w=None, b=None, scale=None, shift=None, eps=1e-6):
    """n"""
    v = normed(h, pre, eps)[0]
    v = v * (1.0 if w is None else w) + (0.0 if b is None else b)
    return v * (1.0 + _rows(scale, seq)) + _rows(shift, seq)


def backward(dh, dn, h, y, seq, G, alpha=1.0, post="none", post_w=None, gate=None, pre="rms",
             w=None, b=None, scale=None, eps=1e-6):
    """Gradients by name, over the rows with seq >= 0."""
    live = seq >= 0
    C = h.shape[1]
    s = seq[live]

    def by_sequence(a):
        out = np.zeros((G, C))
        np.add.at(out, s, a)
        return out

    d = np.zeros((live.sum(), C)) if dh is None else dh[live]
    out = {}
    if dn is not None:
        g = dn[live]
        v, r = normed(h[live], pre, eps)
        wv = 1.0 if w is None else w
        m = 1.0 + _rows(scale, s)
        out["scale"] = by_sequence(g * (v * wv + (0.0 if b is None else b)))
        out["shift"] = by_sequence(g)
        out["weight"] = (g * m * v).sum(axis=0)
        out["bias"] = (g * m * np.ones_like(v)).sum(axis=0)
        d = d + _back(g * m * wv, v, r, pre)
    out["dx"] = np.zeros_like(h)
    out["dx"][live] = alpha * d
    if y is not None:
        gt = 1.0 if gate is None else _rows(gate, s)
        pw = 1.0 if post_w is None else post_w
        q, r = (y[live], None) if post == "none" else normed(y[live], post, eps)
        out["gate"] = by_sequence(d * q * pw)
        out["post_weight"] = (d * gt * q).sum(axis=0)
        e = d * gt * pw
        out["dy"] = np.zeros_like(h)
        out["dy"][live] = e if post == "none" else _back(e, q, r, post)
    return out
