"""Attention of packed sequences with shared key heads and masked keys, in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

q is (Tq, Hq, D), k and v (Tk, Hk, D); ``allowed`` (Tq, Tk) says which keys count for a
query.  A query without one (or with none above -infinity) has o = 0 and lse = -inf.
"""

import numpy as np


def allowed(Tq, Tk, q_offsets=None, kv_offsets=None, kv_lengths=None, key_mask=None):
    """(Tq, Tk) of truth values"""
    def owner(T, offsets):
        g = np.full(T, -1)
        for i in range(len(offsets) - 1):
            g[offsets[i]:offsets[i + 1]] = i
        return g

    q_offsets = [0, Tq] if q_offsets is None else list(q_offsets)
    kv_offsets = [0, Tk] if kv_offsets is None else list(kv_offsets)
    qs, ks = owner(Tq, q_offsets), owner(Tk, kv_offsets)
    ok = (qs[:, None] == ks[None, :]) & (qs >= 0)[:, None]
    if kv_lengths is not None:
        place = np.arange(Tk) - np.asarray(kv_offsets)[np.maximum(ks, 0)]
        ok &= (place < np.asarray(kv_lengths)[np.maximum(ks, 0)])[None, :]
    if key_mask is not None:
        ok &= np.asarray(key_mask, bool)[None, :]
    return ok


def _head(k, h, Hq):
    return k[:, h // (Hq // k.shape[1])]


def scores(q, k, ok, scale):
    """(Hq, Tq, Tk), -inf where a key does not count"""
    Hq = q.shape[1]
    keep = ok.any(axis=0)
    out = np.empty((Hq, q.shape[0], k.shape[0]))
    for h in range(Hq):
        s = q[:, h] @ np.where(keep[:, None], _head(k, h, Hq), 0.0).T * scale
        out[h] = np.where(ok, s, -np.inf)
    return out


def forward(q, k, v, ok, scale):
    """(o, lse)"""
    s = scores(q, k, ok, scale)
    keep = ok.any(axis=0)
    o, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    for h in range(q.shape[1]):
        top = s[h].max(axis=1, initial=-np.inf)
        some = top > -np.inf
        p = np.zeros_like(s[h])
        p[some] = np.exp(s[h][some] - top[some, None])
        total = p.sum(axis=1)
        vals = np.where(keep[:, None], _head(v, h, q.shape[1]), 0.0)
        o[some, h] = (p[some] / total[some, None]) @ vals
        lse[some, h] = top[some] + np.log(total[some])
    return o, lse


def weights(s, lse):
    """p (Hq, Tq, Tk) of scores and the rows' logarithms (Tq, Hq)"""
    l = lse.T[:, :, None]
    return np.where(np.isfinite(l) & (s > -np.inf), np.exp(np.minimum(s - np.where(np.isfinite(l), l, 0.0), 700)), 0.0)


def backward(do, q, k, v, o, lse, ok, scale):
    """(dq, dk, dv) from the forward's o and lse"""
    Hq, Hk = q.shape[1], k.shape[1]
    p = weights(scores(q, k, ok, scale), lse)
    keep = ok.any(axis=0)[:, None]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for h in range(Hq):
        kh, vh = (np.where(keep, _head(t, h, Hq), 0.0) for t in (k, v))
        ds = p[h] * (do[:, h] @ vh.T - (do[:, h] * o[:, h]).sum(axis=1, keepdims=True))
        live = ok.any(axis=1)[:, None]
        dq[:, h] = np.where(live, scale * ds @ kh, 0.0)
        dk[:, h // (Hq // Hk)] += scale * ds.T @ q[:, h]
        dv[:, h // (Hq // Hk)] += p[h].T @ do[:, h]
    return dq, dk, dv
