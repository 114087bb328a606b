"""Head norms with rotation against the float64 oracle, forward and backward, through the
public Python layer.

Gates (from the arithmetic, u = 2^-24 the half step of float32).  A head's sums of D <= 256
elements have 8 additions in a lane and 5 between lanes: off by 13 u of their magnitudes.  So
  r = 1 / sqrt(mean v^2 + eps)    off by 13/2 + 6 < 16 u of itself,
  a normed element                off by 16 u of itself, and for a layer norm by 32 u r max|x| more,
                                  since the mean is off by 16 u of the mean of magnitudes,
  u = x^ w, then a c - b s        off by 24 u of (|a| + |b|) and the layer norm's share,
where (a, b) is bounded by the head's largest element.  The backward adds one such turn before the
norm's formula and sums of two products of D elements: 64 u of the head's largest |g w|, times r,
with (1 + |v| max|v|).  A weight's sum over N heads is off by N u of its magnitudes, beside
what enters.  Results are rounded once: half a step of their type.
"""

import numpy as np
import pytest
import torch

from oracle import heads as O
from wam_asp_w4a4_amd.heads import HeadNorm, head_norm, head_norm_backward

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
EPS = 1e-6


def host(t):
    return None if t is None else t.double().cpu().numpy()


def near(got, want, bound, half):
    off = np.abs(got - want) - (bound + half * (np.abs(want) + bound))
    assert np.isfinite(got).all() and (not off.size or off.max() <= 0), off.max()


class Case:
    def __init__(self, T, Hq, Hk, D, rot=None, norm="rms", layout="pairs", dtype="bf16", positions=None, P=None, weights=True,
                 ld=0, seed=0):
        g = torch.Generator(device=DEV).manual_seed(T * 131 + D * 7 + seed)
        rnd = lambda *s: torch.randn(s, generator=g, device=DEV)
        t = TYPES[dtype]
        rot = D if rot is None else rot
        # one projection's result: queries, keys and something behind them
        self.qkv = (rnd(T, Hq + Hk + 1, D + ld) * 2 + 0.3).to(t)
        self.q = self.qkv[:, :Hq, :D]
        self.k = self.qkv[:, Hq:Hq + Hk, :D] if Hk else None
        self.dq, self.dk = rnd(T, Hq, D).to(t), rnd(T, Hk, D).to(t) if Hk else None
        w = weights and norm != "none"
        P = T + 5 if P is None else P
        angle = torch.rand((P, rot // 2), generator=g, device=DEV) * 6 - 3
        self.kw = dict(norm=norm, layout=layout, eps=EPS, q_weight=1 + 0.3 * rnd(D) if w else None,
                       k_weight=1 + 0.3 * rnd(D) if w and Hk else None,
                       cos=torch.cos(angle) if rot else None, sin=torch.sin(angle) if rot else None,
                       positions=None if positions is None else torch.tensor(positions, dtype=torch.int32, device=DEV))
        self.norm, self.T = norm, T

    def oracle_kw(self, which):
        kw = {n: host(v) if isinstance(v, torch.Tensor) else v for n, v in self.kw.items()}
        w = kw.pop(which + "_weight")
        kw.pop(("k" if which == "q" else "q") + "_weight")
        if kw["positions"] is not None:
            kw["positions"] = kw["positions"].astype(int)
        return dict(w=w, **kw)

    def sides(self):
        return [s for s in (("q", self.q, self.dq), ("k", self.k, self.dk)) if s[1] is not None]

    def scales(self, which, x):
        """(largest |x^ w| of each head with a layer norm's share, r)"""
        v, r = O.normed(x, self.norm, EPS)
        w = self.oracle_kw(which)["w"]
        w = np.ones(x.shape[-1]) if w is None else w
        share = np.abs(x).max(-1, keepdims=True) * r * np.abs(w).max() if self.norm == "layer" else 0.0
        return np.abs(v * w).max(-1, keepdims=True) + share, r, v, w


def check_forward(case, out=None):
    got = head_norm(case.q, case.k, out=out, **case.kw)
    torch.cuda.synchronize()
    for (which, x, _), y in zip(case.sides(), got):
        x = host(x)
        want = O.forward(x, **case.oracle_kw(which))
        near(host(y), want, 2 * 32 * U * case.scales(which, x)[0], HALF[y.dtype])
    return got


def check_backward(case):
    got = head_norm_backward(case.dq, case.dk, case.q, case.k, **case.kw)
    torch.cuda.synchronize()
    for which, x, dy in case.sides():
        kw = case.oracle_kw(which)
        xh, dyh = host(x), host(dy)
        dx, dw = O.backward(dyh, xh, **kw)
        top, r, v, w = case.scales(which, xh)
        g = 2 * np.abs(dyh).max(-1, keepdims=True)          # a turned pair is at most |a| + |b|
        vm = np.abs(v).max(-1, keepdims=True) + (top if case.norm == "layer" else 0.0)
        bound = 0.0 if case.norm == "none" else 64 * U * r * g * np.abs(w).max() * (1 + vm * vm)
        bound = bound + 8 * U * g * np.abs(w).max()
        near(host(getattr(got, "d" + which)), dx, bound, HALF[x.dtype])
        dw_got = getattr(got, which + "_weight")
        if kw["w"] is not None:
            n = x.shape[0] * x.shape[1]
            near(host(dw_got), dw, (n + 64) * U * (g * vm).sum(axis=(0, 1)), 0.0)
        else:
            assert dw_got is None
    return got


SIZES = [  # T, Hq, Hk, D, rot
    (1, 16, 16, 64, 64), (1, 1, 0, 128, 128), (5, 32, 8, 128, 128), (33, 3, 1, 72, 36), (17, 6, 2, 80, 40), (64, 8, 8, 96, 96),
    (7, 5, 3, 2, 2), (9, 4, 4, 30, 14), (3, 2, 2, 256, 128), (130, 12, 4, 34, 0), (2, 70, 33, 64, 32), (3000, 2, 1, 48, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["pairs", "halves"])
@pytest.mark.parametrize("T, Hq, Hk, D, rot", SIZES)
def test_parity(T, Hq, Hk, D, rot, layout, dtype):
    for norm in ("rms", "layer", "none"):
        print(f"heads T={T} Hq={Hq} Hk={Hk} D={D} rot={rot} {layout} {dtype} {norm}", flush=True)
        case = Case(T, Hq, Hk, D, rot, norm, layout, dtype)
        check_forward(case)
        check_backward(case)


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_other_types_strides_and_no_weights(norm):
    case = Case(40, 6, 2, 72, 40, norm, "halves", "bf16", weights=False, ld=3)   # elements at odd places
    check_forward(case, "f32")
    check_backward(case)
    case = Case(40, 6, 2, 72, 40, norm, "pairs", "f32", ld=1)
    check_forward(case, "bf16")
    # gradients of another type than the inputs', by head first
    case.dq = case.dq.to(torch.bfloat16).transpose(0, 1).contiguous().transpose(0, 1)
    case.dk = case.dk.to(torch.bfloat16)
    check_backward(case)
    # one head for all tokens, and one token's row for all heads: broadcast inputs are read as they are
    case.q = case.q[:1, :1].expand(40, 6, 72)
    check_forward(case)
    check_backward(case)


def test_positions_and_padding():
    pos = [3, 0, -1, 7, 8, 2 ** 31 - 1, -2 ** 31, 7]   # tables of 8 positions
    for dtype in ("bf16", "f32"):
        case = Case(8, 4, 2, 64, 64, "layer", "halves", dtype, pos, P=8)
        check_forward(case)
        check_backward(case)
        dead = torch.tensor([2, 4, 5, 6], device=DEV)
        for t in head_norm(case.q, case.k, **case.kw) + head_norm_backward(case.dq, case.dk, case.q, case.k, **case.kw)[:2]:
            assert not t[dead].any()
        # given outputs keep their padding rows
        outs = [torch.full_like(t, 7.0) for t in (case.q, case.k)]
        got = head_norm(case.q, case.k, q_out=outs[0], k_out=outs[1], **case.kw)
        assert got[0] is outs[0] and got[1] is outs[1]
        assert all((t[dead] == 7.0).all() for t in outs)
        want = head_norm(case.q, case.k, **case.kw)
        live = torch.tensor([0, 1, 3, 7], device=DEV)
        assert all(torch.equal(a[live], b[live]) for a, b in zip(outs, want))
        grads = [torch.full_like(t, 7.0) for t in (case.q, case.k)]
        head_norm_backward(case.dq, case.dk, case.q, case.k, dq_in=grads[0], dk_in=grads[1], **case.kw)
        assert all((t[dead] == 7.0).all() for t in grads)


def test_padding_rows_hold_anything():
    case = Case(6, 4, 2, 64, 64, "rms", "pairs", "bf16", [0, 1, -1, 2, 3, 4])
    want = head_norm_backward(case.dq, case.dk, case.q, case.k, **case.kw)
    for t in (case.qkv, case.dq, case.dk):
        t[2] = float("nan")
    got = head_norm_backward(case.dq, case.dk, case.q, case.k, **case.kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not any(t.isnan().any() for t in head_norm(case.q, case.k, **case.kw))


def test_a_nan_reaches_its_own_head():
    case = Case(6, 4, 2, 128, 128, "layer", "halves", "f32")
    want = head_norm(case.q, case.k, **case.kw)
    case.qkv[3, 1, 77] = float("nan")
    case.qkv[4, 5, 0] = float("inf")
    got = head_norm(case.q, case.k, **case.kw)
    bad = [torch.zeros_like(w, dtype=torch.bool) for w in want]
    bad[0][3, 1] = bad[1][4, 1] = True
    for g, w, b in zip(got, want, bad):
        assert torch.equal(g[~b], w[~b]) and g[b].isnan().all()


def test_in_place_and_zero_tokens():
    for layout in ("pairs", "halves"):
        case = Case(50, 8, 2, 96, 48, "rms", layout, "bf16")
        want = head_norm(case.q, case.k, **case.kw)
        back = head_norm_backward(case.dq, case.dk, case.q, case.k, **case.kw)
        head_norm_backward(case.dq, case.dk, case.q, case.k, dq_in=case.dq, dk_in=case.dk, **case.kw)
        assert torch.equal(case.dq, back.dq) and torch.equal(case.dk, back.dk)
        head_norm(case.q, case.k, q_out=case.q, k_out=case.k, **case.kw)
        assert torch.equal(case.q, want[0]) and torch.equal(case.k, want[1])
    case = Case(0, 4, 2, 64, 64, "rms", "pairs", "f32", P=3)
    q, k = head_norm(case.q, case.k, **case.kw)
    g = head_norm_backward(case.dq, case.dk, case.q, case.k, **case.kw)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64) and not g.q_weight.any() and not g.k_weight.any()


def test_same_bits_and_wanted_gradients_alone():
    case = Case(2100, 8, 2, 128, 128, "rms", "halves", "bf16")
    want = head_norm_backward(case.dq, case.dk, case.q, case.k, **case.kw)
    for need in (("dq", "dk", "q_weight", "k_weight"), ("dq",), ("k_weight",), ("q_weight", "dk"), ("dk", "k_weight")):
        got = head_norm_backward(case.dq, case.dk, case.q, case.k, need=iter(need), **case.kw)
        for name, a, b in zip(want._fields, got, want):
            assert (a is None) == (name not in need)
            assert a is None or torch.equal(a, b), name
    # what is not needed is not read
    got = head_norm_backward(None, case.dk, case.q, case.k, need=("dk",), **case.kw)
    assert torch.equal(got.dk, want.dk)


def test_rows_past_2_to_the_31_elements():
    T, H, D = 1100, 2, 64
    ld = 2 ** 21
    big = torch.empty(T * ld, dtype=torch.bfloat16, device=DEV)
    q = torch.as_strided(big, (T, H, D), (ld, D, 1))
    q.copy_(torch.randn((T, H, D), device=DEV))
    case = Case(T, H, 0, D)
    want = head_norm(q.contiguous(), **case.kw)[0]
    assert torch.equal(head_norm(q, **case.kw)[0], want)
    assert torch.equal(head_norm(q, q_out=q, **case.kw)[0], want)
    del big, q


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_module_gradients(dtype):
    B, T, Hq, Hk, D = 3, 20, 4, 2, 64
    t = TYPES[dtype]
    torch.manual_seed(3)
    m = HeadNorm(D, "layer", "halves", EPS, DEV)
    with torch.no_grad():
        for p in m.parameters():
            p.add_(torch.randn_like(p) * 0.1)
    case = Case(T, 1, 0, D)
    cos, sin = case.kw["cos"], case.kw["sin"]
    pos = torch.randint(-1, T, (B, T), dtype=torch.int32, device=DEV)
    q = torch.randn((B, T, Hq, D), device=DEV).to(t).requires_grad_()
    k = torch.randn((B, T, Hk, D), device=DEV).to(t).requires_grad_()
    gq, gk = torch.randn_like(q), torch.randn_like(k)
    for positions in (pos, pos[0], None):
        y, z = m(q, k, cos, sin, positions)
        assert y.shape == q.shape and z.shape == k.shape and y.dtype == t
        got = torch.autograd.grad([y, z], [q, k, m.q_weight, m.k_weight], [gq, gk])
        at = torch.arange(T, dtype=torch.int32, device=DEV) if positions is None else positions
        flat = at.expand(B, T).reshape(-1).contiguous()
        want = head_norm_backward(gq.flatten(0, 1), gk.flatten(0, 1), q.detach().flatten(0, 1), k.detach().flatten(0, 1), norm="layer",
                                  layout="halves", eps=EPS, q_weight=m.q_weight.detach(), k_weight=m.k_weight.detach(), cos=cos,
                                  sin=sin, positions=flat)
        for a, b in zip(got, want):
            assert torch.equal(a.reshape(b.shape), b)
    # one result alone: the other's gradients are zeros, not errors
    g = torch.autograd.grad(m(q, k, cos, sin)[0].float().sum(), [q, k, m.q_weight, m.k_weight])
    assert g[0].any() and not g[1].any() and not g[3].any()
    with torch.no_grad():
        assert torch.equal(m(q, k, cos, sin)[0], m(q, None, cos, sin)[0])


def test_gradients_are_differences():
    case = Case(6, 2, 1, 32, 16, "layer", "pairs", "f32")
    got = head_norm_backward(case.dq, case.dk, case.q, case.k, **case.kw)
    kw = case.oracle_kw("q")
    x, dy, r = host(case.q), host(case.dq), np.random.default_rng(0)
    for _ in range(4):
        d = r.normal(size=x.shape)
        h = 1e-6
        diff = ((O.forward(x + h * d, **kw) - O.forward(x - h * d, **kw)) * dy).sum() / (2 * h)
        # differences: h^2 and 1e-16 / h of the value; the kernel's own bound is above both
        g = host(got.dq)
        assert abs((g * d).sum() - diff) <= 1e-4 * (np.abs(g) * np.abs(d)).sum() * 1e-1


def test_streams_graphs_and_captures():
    case = Case(300, 8, 2, 128, 128, "rms", "halves", "bf16")
    want = (*head_norm(case.q, case.k, **case.kw), *head_norm_backward(case.dq, case.dk, case.q, case.k, **case.kw))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = (*head_norm(case.q, case.k, stream=side.cuda_stream, **case.kw),
           *head_norm_backward(case.dq, case.dk, case.q, case.k, stream=side.cuda_stream, **case.kw))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (*head_norm(case.q, case.k, **case.kw), *head_norm_backward(case.dq, case.dk, case.q, case.k, **case.kw))
    for i in range(4):
        case.qkv.copy_(torch.randn_like(case.qkv) * (i + 1))
        want = (*head_norm(case.q, case.k, **case.kw), *head_norm_backward(case.dq, case.dk, case.q, case.k, **case.kw))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    m = HeadNorm(128, device=DEV)
    with pytest.raises(RuntimeError, match="capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            m(case.q)
    with pytest.raises(RuntimeError, match="forward-mode"):
        with torch.autograd.forward_ad.dual_level():
            m(torch.autograd.forward_ad.make_dual(case.q.contiguous(), case.q.contiguous()))
