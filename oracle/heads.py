"""The norms of queries and keys, head by head, with the rotation by positions, in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

x is (T, H, D).  u = norm(x) w over the last axis ('rms', 'layer' or 'none'); the first
2 P elements of u are pairs, turned by the angles whose cosines and sines are the rows
``positions`` of (positions, P) tables.  'pairs': pair i is (2i, 2i + 1); 'halves': (i, i + P).
A token whose position is outside the tables has zeros, and adds nothing to a gradient.
"""

import numpy as np


def _indices(P, layout):
    """(first, second) elements of the pairs"""
    i = np.arange(P)
    return (2 * i, 2 * i + 1) if layout == "pairs" else (i, i + P)


def _turn(u, c, s, layout):
    """u with its pairs turned; c, s: (T, P)."""
    first, second = _indices(c.shape[1], layout)
    y = u.copy()
    a, b = u[..., first], u[..., second]
    c, s = c[:, None], s[:, None]
    y[..., first] = a * c - b * s
    y[..., second] = a * s + b * c
    return y


def normed(x, kind, eps):
    if kind == "none":
        return x, np.ones(x.shape[:-1] + (1,))
    if kind == "layer":
        x = x - x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r, r


def _tables(T, cos, sin, positions):
    """(live tokens, their cosines, their sines)"""
    if cos is None:
        return np.ones(T, bool), np.zeros((T, 0)), np.zeros((T, 0))
    p = np.arange(T) if positions is None else np.asarray(positions)
    live = (p >= 0) & (p < cos.shape[0])
    at = np.where(live, p, 0)
    return live, np.asarray(cos, np.float64)[at], np.asarray(sin, np.float64)[at]


def forward(x, norm="rms", w=None, cos=None, sin=None, positions=None, layout="pairs", eps=1e-6):
    live, c, s = _tables(x.shape[0], cos, sin, positions)
    u = normed(x, norm, eps)[0] * (1.0 if w is None else w)
    y = _turn(u, c, s, layout)
    y[~live] = 0.0
    return y


def backward(dy, x, norm="rms", w=None, cos=None, sin=None, positions=None, layout="pairs", eps=1e-6):
    """(dx, dw)"""
    live, c, s = _tables(x.shape[0], cos, sin, positions)
    g = _turn(np.where(live[:, None, None], dy, 0.0), c, -s, layout)
    v, r = normed(x, norm, eps)
    v = np.where(live[:, None, None], v, 0.0)
    dw = (g * v).sum(axis=(0, 1))
    g = g * (1.0 if w is None else w)
    if norm != "none":
        d = g - v * (g * v).mean(-1, keepdims=True)
        if norm == "layer":
            d = d - g.mean(-1, keepdims=True)
        g = d * r
    g[~live] = 0.0
    return g, dw
