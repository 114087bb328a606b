"""The 8-bit format with one power-of-two scale for each block of 128, and the
linear layer on it, in plain NumPy.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

A block of 128 consecutive elements along the contracted axis shares the scale
S = 2^k, the smallest power of two with k >= -126 and max|v| / S <= 448, the
maximum over its finite elements; an element is E4M3FN(v / S), ties to even.  NaN
and infinities take the NaN code with their sign.  A weight's blocks are
128 x 128.  v / S is formed in float64, where it is exact.

    y = Q(x) Q(W)^T + b
    dx = Q(dy) Q(W),  dW = Q(dy^T) Q(x^T)^T,  db = the sum of dy's rows
"""

import numpy as np

from .formats import E4M3_VALUES

BLOCK = 128
_GRID = E4M3_VALUES[:0x7F]          # the non-negative values, code = index


def _codes(q):
    """Codes of quotients |q| <= 448 (or NaN): the nearest grid value, ties to the even code."""
    a = np.abs(q)
    ok = np.isfinite(a)
    a = np.where(ok, a, 0.0)
    hi = np.clip(np.searchsorted(_GRID, a), 0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _GRID[lo], _GRID[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(ok, code, 0x7F)
    return (code | (np.signbit(q).astype(np.int64) << 7)).astype(np.uint8)


def _exponent(top):
    """k of each block's scale, from comparisons of exact values."""
    _, e = np.frexp(top)
    k = e - 9
    k = k + (top > 448.0 * np.exp2(k.astype(np.float64)))
    return np.maximum(np.where(top == 0, -126, k), -126).astype(np.int64)


def quantize(v, square=False):
    """(codes rows x P uint8, scale bytes rows x P/128 uint8) of a matrix."""
    v = np.asarray(v, np.float64)
    rows, cols = v.shape
    pr = -(-rows // BLOCK) * BLOCK if square else rows
    pc = -(-cols // BLOCK) * BLOCK
    p = np.zeros((pr, pc))
    p[:rows, :cols] = v
    fin = np.where(np.isfinite(p), np.abs(p), 0.0).reshape(pr, pc // BLOCK, BLOCK).max(axis=2)
    if square:
        fin = fin.reshape(pr // BLOCK, BLOCK, -1).max(axis=1).repeat(BLOCK, axis=0)
    k = _exponent(fin)
    unit = np.exp2(k.astype(np.float64)).repeat(BLOCK, axis=1)
    with np.errstate(invalid="ignore"):
        codes = _codes(p / unit)
    return codes[:rows], (k + 127).astype(np.uint8)[:rows]


def values(codes, scale_bytes, cols):
    """float64 values of codes under their block scales."""
    s = np.exp2(scale_bytes.astype(np.float64) - 127).repeat(BLOCK, axis=1)
    return (E4M3_VALUES[codes] * s)[:, :cols]


def held(v, square=False):
    """v as the format holds it."""
    return values(*quantize(v, square), np.asarray(v).shape[1])


def layout_scales(scale_bytes):
    """Scale bytes rows x blocks -> the device layout [groups of 4][rows][4], padded with 127."""
    rows, nb = scale_bytes.shape
    p = np.full((rows, -(-nb // 4) * 4), 127, np.uint8)
    p[:, :nb] = scale_bytes
    return np.ascontiguousarray(p.reshape(rows, -1, 4).transpose(1, 0, 2))


def forward(x, w, b=None):
    y = held(x) @ held(w, square=True).T
    return y if b is None else y + b


def backward(dy, x, w):
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    return (held(dy) @ held(w, square=True), held(dy.T) @ held(x.T).T, dy.sum(axis=0))
