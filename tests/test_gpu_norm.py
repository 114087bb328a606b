"""The gated norms against the float64 oracle, forward and backward, through the
public Python layer.

Gates (from the arithmetic, u = 2^-24 the half step of float32):
* a row's sum has at most 32 additions in a lane, 6 in a wave and 8 between waves one
  after the other, so it is off by at most 46 u of the sum of magnitudes; with the few
  roundings of each further step, a normed value v is off by 64 u (1 + |v| + r mean|h|):
  r from the sum of squares, and for a layer norm the mean of the row.  Every later
  factor and addition keeps that relative to the magnitudes that enter it;
* h is rounded once to x's type (half a step); n is judged against the pre norm of the h
  that the device stored, as it is defined, and rounded once to its own type;
* column sums over M rows are off by M u of the sum of magnitudes, beside what enters.
"""

import numpy as np
import pytest
import torch

from oracle import fp8 as OF
from oracle import norm as O
from wam_asp_w4a4_amd import binding as B
from wam_asp_w4a4_amd.fp8 import Fp8Layer, Fp8Tensor, quantize
from wam_asp_w4a4_amd.norm import GatedNorm, gated_norm, gated_norm_backward

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
EPS = 1e-6


def host(t):
    return None if t is None else t.double().cpu().numpy()


def near(got, want, bound, half, live=None):
    bound = np.broadcast_to(bound, want.shape)
    off = np.abs(got - want) - (bound + half * (np.abs(want) + bound))
    if live is not None:
        off = off[live]
    assert not off.size or off.max() <= 0, off.max()


class Case:
    def __init__(self, M, C, dtype, post, pre, tables, offsets, affine=True, alpha=0.7, ld=0):
        g = torch.Generator(device=DEV).manual_seed(M * 131 + C)
        rnd = lambda *s: torch.randn(s, generator=g, device=DEV)
        t = TYPES[dtype]
        self.M, self.C, self.dtype, self.t = M, C, dtype, t
        self.seq = O.sequences(M, offsets)
        self.live = self.seq >= 0
        self.G = 1 if offsets is None else len(offsets) - 1
        wide = lambda: torch.empty((M, C + ld), dtype=t, device=DEV)[:, :C].copy_(rnd(M, C) * 2 + 0.5)
        self.x, self.y, self.dh, self.dn = wide(), wide(), wide(), wide()
        table = rnd(self.G, 3, C) * 0.5
        self.kw = dict(alpha=alpha, post=post, pre=pre, eps=EPS,
                       post_weight=1 + 0.2 * rnd(C) if post != "none" else None,
                       gate=table[:, 0] if tables else None,
                       scale=table[:, 1] if tables and pre != "none" else None,
                       shift=table[:, 2] if tables and pre != "none" else None,
                       weight=1 + 0.2 * rnd(C) if affine and pre != "none" else None,
                       bias=rnd(C) if affine and pre != "none" else None,
                       offsets=None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV))

    def host(self, name):
        return host(self.kw[name])

    def check_forward(self, h, n):
        k, live = self.kw, self.live
        x, y = host(self.x), host(self.y)
        gate = np.abs(O._rows(k["gate"].double().cpu().numpy(), self.seq)) if k["gate"] is not None else 1.0
        want = O.stream(x, y, self.seq, k["alpha"], k["post"], self.host("post_weight"), self.host("gate"), EPS)
        q, r = (y, 1.0) if k["post"] == "none" else O.normed(y, k["post"], EPS)
        pw = 1.0 if k["post_weight"] is None else np.abs(self.host("post_weight"))
        bound = U * (4 * np.abs(k["alpha"] * x) + gate * pw * (8 * np.abs(q) if k["post"] == "none" else
                     64 * (1 + np.abs(q) + r * np.abs(y).mean(axis=1, keepdims=True))))
        got = host(h)
        near(got, want, bound, HALF[self.dtype], live)
        if n is None:
            return
        v, r = O.normed(got, k["pre"], EPS)
        want = O.prenorm(got, self.seq, k["pre"], self.host("weight"), self.host("bias"), self.host("scale"),
                         self.host("shift"), EPS)
        w = 1.0 if k["weight"] is None else np.abs(self.host("weight"))
        b = 0.0 if k["bias"] is None else np.abs(self.host("bias"))
        m = 1.0 + (np.abs(O._rows(self.host("scale"), self.seq)) if k["scale"] is not None else 0.0)
        s = np.abs(O._rows(self.host("shift"), self.seq)) if k["shift"] is not None else 0.0
        bound = U * (64 * (1 + np.abs(v) + r * np.abs(got).mean(axis=1, keepdims=True)) * w * m + 8 * (b * m + s))
        near(host(n), want, bound, HALF["bf16" if n.dtype == torch.bfloat16 else "f32"], live)


SEQ = [0, 5, 5, 6, 29]            # an empty sequence, one of one row, padding behind
SIZES = [(1, 1), (3, 7), (40, 128), (33, 512), (40, 1000), (33, 1024), (33, 1001), (30, 2048), (31, 4096),
         (30, 5000), (30, 9001), (30, 16384)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,C", SIZES)
def test_forward_sizes(M, C, dtype):
    print(f"norm {M}x{C} {dtype}", flush=True)
    c = Case(M, C, dtype, "rms", "layer", True, SEQ if M >= 30 else None)
    h, n = gated_norm(c.x, c.y, **c.kw)
    assert n.dtype == c.t
    c.check_forward(h, n)
    again = gated_norm(c.x, c.y, **c.kw)
    live = torch.from_numpy(c.live).to(DEV)
    assert torch.equal(again[0][live], h[live]) and torch.equal(again[1][live], n[live])


@pytest.mark.parametrize("tables", [False, True])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
def test_forward_kinds(pre, post, tables):
    for offsets, ld, affine, out in ((None, 0, True, None), (SEQ, 13, False, "f32"), ([2, 8, 20], 8, True, "bf16")):
        c = Case(32, 328, "bf16", post, pre, tables, offsets, affine, ld=ld)
        h, n = gated_norm(c.x, c.y, out=None if pre == "none" else out, **c.kw)
        assert (n is None) == (pre == "none")
        c.check_forward(h, n)


def test_rows_of_no_sequence_are_left_and_buffers_are_used():
    c = Case(40, 300, "bf16", "rms", "rms", True, [3, 9, 9, 30], ld=4)
    h, n = torch.full_like(c.x, 5.0), torch.full((40, 320), 6.0, device=DEV)
    got = gated_norm(c.x, c.y, h=h, n=n[:, :300], **c.kw)
    assert got[0] is h
    c.check_forward(h, got[1])
    dead = torch.from_numpy(~c.live).to(DEV)
    assert (h[dead] == 5).all() and (n[dead] == 6).all() and (n[:, 300:] == 6).all()
    # padding may hold anything
    c.x[dead], c.y[dead] = float("nan"), float("inf")
    again = gated_norm(c.x, c.y, out="f32", **c.kw)
    assert torch.equal(again[0][~dead], h[~dead]) and torch.equal(again[1][~dead], n[:, :300][~dead])
    # h in place of x, and of y
    for name in ("x", "y"):
        x, y = c.x.clone(), c.y.clone()
        out = {"x": x, "y": y}[name]
        gated_norm(x, y, h=out, **c.kw)
        assert torch.equal(out[~dead], h[~dead])


def test_special_values():
    c = Case(8, 256, "f32", "layer", "rms", False, None)
    x, y = c.x.clone(), c.y.clone()
    x[1], y[1] = 0.0, 0.0                       # an empty row: 0 / sqrt(eps)
    y[2] = 3.0                                  # a constant row: its layer norm is 0
    y[3, 7], x[4, 9] = float("nan"), float("inf")
    h, n = gated_norm(x, y, alpha=1.0, post="layer", pre="rms")
    assert not h[1].any() and not n[1].any() and torch.equal(h[2], x[2])
    assert torch.isnan(n[[3, 4]]).any(dim=1).all()
    assert torch.isfinite(n[[0, 1, 2, 5, 6, 7]]).all()
    # a mean far above the deviation: no difference of large squares
    big = torch.randn((4, 1024), device=DEV) + 4096.0
    _, n = gated_norm(big, pre="layer")
    near(host(n), O.normed(host(big), "layer", EPS)[0], 64 * U * 4100, U)


@pytest.mark.parametrize("M,C", [(1, 1), (9, 100), (40, 128), (33, 640), (30, 1001), (40, 1536), (30, 5000)])
def test_eight_bit_result(M, C):
    """The codes are those of the row quantiser for the float32 n, bit for bit."""
    print(f"eight bit {M}x{C}", flush=True)
    c = Case(M, C, "bf16", "none", "layer", True, SEQ if M >= 30 else None)
    _, n = gated_norm(c.x, c.y, out="f32", **c.kw)
    h, q = gated_norm(c.x, c.y, out="fp8", **c.kw)
    live = torch.from_numpy(c.live).to(DEV)
    want = quantize(n)
    assert torch.equal(q.codes[live], want.codes[live]) and torch.equal(q.scales[:, live], want.scales[:, live])
    # into the caller's tensor: rows of no sequence keep their codes
    mine = Fp8Tensor.empty(M, C, DEV)
    mine.codes.fill_(9), mine.scales.fill_(8)
    gated_norm(c.x, c.y, n=mine, **c.kw)
    assert torch.equal(mine.codes[live], want.codes[live])
    assert (mine.codes[~live] == 9).all() and (mine.scales[:, ~live] == 8).all()


@pytest.mark.parametrize("M", [3, 200])
def test_block_end_to_next_projection(M):
    """A run as it is used: norms, 8-bit codes, the linear layer that reads them."""
    C, N = 640, 300
    c = Case(M, C, "bf16", "rms", "layer", True, None)
    w = torch.randn((N, C), device=DEV) / C ** 0.5
    layer = Fp8Layer.pack(w, torch.randn(N, device=DEV))
    h, q = gated_norm(c.x, c.y, out="fp8", **c.kw)
    y = layer.forward(q, "f32")
    qv, wv = host(q.dequantize()), OF.held(host(w), square=True)
    near(host(y), qv @ wv.T + host(layer.bias), C * 2 * U * (np.abs(qv) @ np.abs(wv).T + 1), U)
    # against the unquantised n: half a step of E4M3 for each element
    _, n = gated_norm(c.x, c.y, out="f32", **c.kw)
    nv = host(n)
    step = np.maximum(np.abs(nv) / 16, np.abs(nv).max() / 448 / 512)
    assert (np.abs(host(y) - (nv @ wv.T + host(layer.bias))) <= step @ np.abs(wv).T + 1e-4).all()


BACK = [(1, 1, "f32"), (5, 7, "f32"), (40, 128, "bf16"), (33, 512, "f32"), (70, 1000, "bf16"), (33, 1001, "f32"),
        (30, 2048, "bf16"), (31, 4096, "bf16"), (30, 5000, "f32"), (30, 9001, "bf16"), (30, 16384, "bf16"),
        (5000, 64, "f32"), (1500, 1100, "bf16")]


def check_backward(c, y=True, dh=True):
    k, C, M = c.kw, c.C, c.M
    yt, dht = (c.y if y else None), (c.dh if dh else None)
    dx0, dy0 = torch.full_like(c.x, 5.0), torch.full_like(c.x, 6.0) if y else None
    dn = c.dn if k["pre"] != "none" else None
    got = gated_norm_backward(dht, dn, c.x, yt, dx=dx0, dy=dy0, **k)
    want = O.backward(host(dht), host(dn), host(c.x), host(yt), c.seq, c.G, k["alpha"], k["post"], c.host("post_weight"),
                      c.host("gate"), k["pre"], c.host("weight"), c.host("bias"), c.host("scale"), EPS)
    # magnitudes: of the gradient that reaches h through the pre norm, and onwards to y
    h, d, e = host(c.x), host(dn), np.zeros((M, C)) if dht is None else np.abs(host(dht))
    live = c.live
    sums = {}
    if dn is not None:
        v, r = O.normed(h, k["pre"], EPS)
        w = 1.0 if k["weight"] is None else np.abs(c.host("weight"))
        m = 1.0 + (np.abs(O._rows(c.host("scale"), c.seq)) if k["scale"] is not None else 0.0)
        g = np.abs(d) * w * m
        spread = 1 + np.abs(v) + r * np.abs(h).mean(axis=1, keepdims=True)
        mean = lambda a: a.mean(axis=1, keepdims=True)
        e = e + r * (g + mean(g) + spread * mean(g * spread))
        b = 0.0 if k["bias"] is None else np.abs(c.host("bias"))
        sums["scale"], sums["shift"] = np.abs(d) * (spread * w + b), np.abs(d)
        sums["weight"], sums["bias"] = np.abs(d) * m * spread, np.abs(d) * m
    rows = 256 * U   # three row sums one after the other
    near(host(got.dx), want["dx"], abs(k["alpha"]) * rows * e, HALF[c.dtype], live)
    assert (got.dx[torch.from_numpy(~live).to(DEV)] == 5).all()
    if y:
        q, r = (np.abs(host(c.y)), 1.0) if k["post"] == "none" else O.normed(host(c.y), k["post"], EPS)
        spread = np.abs(q) if k["post"] == "none" else 1 + np.abs(q) + r * np.abs(host(c.y)).mean(axis=1, keepdims=True)
        gt = 1.0 if k["gate"] is None else np.abs(O._rows(c.host("gate"), c.seq))
        pw = 1.0 if k["post_weight"] is None else np.abs(c.host("post_weight"))
        sums["gate"], sums["post_weight"] = e * spread * pw, e * spread * gt
        f = e * gt * pw
        if k["post"] != "none":
            f = r * (f + f.mean(axis=1, keepdims=True) + spread * (f * spread).mean(axis=1, keepdims=True))
        near(host(got.dy), want["dy"], 3 * rows * f, HALF[c.dtype], live)
        assert (got.dy[torch.from_numpy(~live).to(DEV)] == 6).all()
    for name, mass in sums.items():
        t = getattr(got, name)
        if t is None:
            assert k[name] is None
            continue
        assert t.dtype == torch.float32 and t.shape == k[name].shape
        by = np.zeros((c.G, C))
        np.add.at(by, c.seq[live], np.broadcast_to(mass, (M, C))[live])
        bound = (rows * 3 + (M + 16) * U) * (by if t.dim() == 2 else by.sum(axis=0))
        near(host(t), want[name], bound, U)
    return got


@pytest.mark.parametrize("M,C,dtype", BACK)
def test_backward_sizes(M, C, dtype):
    print(f"norm backward {M}x{C} {dtype}", flush=True)
    c = Case(M, C, dtype, "layer", "rms", True, SEQ if M >= 30 else None)
    first = check_backward(c)
    again = gated_norm_backward(c.dh, c.dn, c.x, c.y, **c.kw)
    assert all(torch.equal(a, b) for a, b in zip(first[2:], again[2:]))


@pytest.mark.parametrize("tables", [False, True])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
def test_backward_kinds(pre, post, tables):
    for offsets, ld, affine in ((None, 0, True), (SEQ, 13, False), ([2, 8, 20], 8, True)):
        check_backward(Case(32, 328, "bf16", post, pre, tables, offsets, affine, ld=ld))
    if pre != "none":
        c = Case(32, 328, "f32", post, pre, tables, SEQ)
        check_backward(c, dh=False)
        c.dn = c.dn.bfloat16()
        check_backward(c)
        if post == "none" and not tables:
            check_backward(c, y=False)


def test_backward_against_differences():
    """float32 differences over a step of 2^-6: off by its square times the third
    derivative (below 1 in these units) and by 2^-24 of the loss's terms over the step."""
    c = Case(24, 96, "f32", "rms", "layer", True, [0, 7, 7, 20])
    live = torch.from_numpy(c.live).to(DEV)[:, None].double()

    def loss(x, y, **over):
        h, n = gated_norm(x, y, **{**c.kw, **over})
        return ((h.double() * c.dh.double() + n.double() * c.dn.double()).nan_to_num() * live).sum().item()

    h, _ = gated_norm(c.x, c.y, **c.kw)
    g = gated_norm_backward(c.dh, c.dn, h, c.y, **c.kw)
    step = 2.0 ** -6
    for name in ("x", "y", "gate", "scale", "shift", "weight", "bias", "post_weight"):
        v = {"x": c.x, "y": c.y}.get(name, c.kw.get(name))
        grad = {"x": g.dx, "y": g.dy}.get(name)
        grad = getattr(g, name) if grad is None else grad
        d = torch.randn_like(v).contiguous()
        if name in ("x", "y"):
            d = d * live.float()
            ends = [loss(*((v + s * step * d, c.y) if name == "x" else (c.x, v + s * step * d))) for s in (1, -1)]
        else:
            table = lambda s: torch.stack([v + s * step * d] * 3, 1)[:, 0] if v.dim() == 2 else v + s * step * d
            ends = [loss(c.x, c.y, **{name: table(s)}) for s in (1, -1)]
        diff = (ends[0] - ends[1]) / (2 * step)
        want = ((grad * live.float() if name in ("x", "y") else grad).double() * d.double()).sum().item()
        mass = (c.dn.abs().double() * live).sum().item()
        assert abs(diff - want) <= mass * (step ** 2 + 2.0 ** -24 * 64 / step), (name, diff, want)


def test_no_rows():
    x = torch.empty((0, 64), device=DEV)
    h, n = gated_norm(x, x, weight=torch.ones(64, device=DEV))
    assert h.shape == n.shape == (0, 64)
    g = gated_norm_backward(x, x, x, x, weight=torch.ones(64, device=DEV))
    assert not g.weight.any()


def test_captured_calls_replay_like_eager_ones():
    c = Case(64, 1024, "bf16", "rms", "layer", True, [0, 20, 20, 60])
    live = torch.from_numpy(c.live).to(DEV)
    ws = torch.empty(B.asp_norm_gate_backward_workspace_bytes(64, 1024, 3), dtype=torch.uint8, device=DEV)
    run = lambda: (*gated_norm(c.x, c.y, **c.kw), gated_norm_backward(c.dh, c.dn, c.x, c.y, workspace=ws, **c.kw))
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, n, g = run()
    for i in range(4):
        for t in (c.x, c.y, c.dh, c.dn):
            t.copy_(torch.randn_like(t) * (i + 1))
        c.kw["offsets"].copy_(torch.tensor([0, 20 - i, 20 + i, 60], dtype=torch.int32))
        wh, wn, wg = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h[live], wh[live]) and torch.equal(n[live], wn[live])
        assert torch.equal(g.dx[live], wg.dx[live]) and torch.equal(g.dy[live], wg.dy[live])
        assert all(torch.equal(a, b) for a, b in zip(g[2:], wg[2:]))


def test_module_trains():
    """GatedNorm under autograd gives gated_norm_backward's gradients."""
    m = GatedNorm(160, post="rms", pre="layer").to(DEV)
    with torch.no_grad():
        for p in m.parameters():
            p.add_(torch.randn_like(p) * 0.1)
    x = torch.randn((2, 5, 160), device=DEV, requires_grad=True)
    y = torch.randn((2, 5, 160), device=DEV, requires_grad=True)
    gate = torch.randn((2, 160), device=DEV, requires_grad=True)
    off = torch.tensor([0, 5, 10], dtype=torch.int32, device=DEV)
    h, n = m(x, y, gate=gate, offsets=off)
    dh, dn = torch.randn_like(h), torch.randn_like(n)
    torch.autograd.backward([h, n], [dh, dn])
    g = gated_norm_backward(dh.view(10, 160), dn.view(10, 160), h.detach().view(10, 160), y.detach().view(10, 160),
                            post="rms", pre="layer", post_weight=m.post_weight.detach(), gate=gate.detach(),
                            weight=m.weight.detach(), bias=m.bias.detach(), offsets=off)
    assert torch.equal(x.grad.view(10, 160), g.dx) and torch.equal(y.grad.view(10, 160), g.dy)
    assert torch.equal(gate.grad, g.gate) and torch.equal(m.weight.grad, g.weight)
    assert torch.equal(m.bias.grad, g.bias) and torch.equal(m.post_weight.grad, g.post_weight)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,C,offsets", [(9, 40, [2, 2, 5]), (40, 200, [0, 11, 33]), (7, 1100, [7, 7, 7]),
                                         (5000, 130, [700, 1300, 4200]), (6, 8300, [1, 4, 5])])
def test_rows_of_no_sequence_are_zeros_in_tensors_made_here(M, C, offsets, dtype):
    print(f"zeros {M}x{C} {dtype} {offsets}", flush=True)
    c = Case(M, C, dtype, "rms", "layer", True, offsets)
    dead = torch.from_numpy(~c.live).to(DEV)
    for out in ("f32", "bf16", "fp8"):
        trash = [torch.full((M, C), float("nan"), device=DEV) for _ in range(4)]
        del trash                                            # what the allocator hands out next
        h, n = gated_norm(c.x, c.y, out=out, **c.kw)
        if out == "fp8":
            assert (n.scales[:, dead] == 127).all() and not n.codes[dead].any()
            n = n.dequantize()
        assert not h[dead].any() and not n[dead].any()
        given = torch.full((M, C), 5.0, dtype=c.t, device=DEV)
        assert gated_norm(c.x, c.y, h=given, **c.kw)[0] is given
        assert (given[dead] == 5).all() and torch.equal(given[~dead], h[~dead])
    g = gated_norm_backward(c.dh, c.dn, h, c.y, **c.kw)
    assert not g.dx[dead].any() and not g.dy[dead].any()
    mine = torch.full((M, C), 5.0, dtype=c.t, device=DEV)
    assert torch.equal(gated_norm_backward(c.dh, c.dn, h, c.y, dy=mine, **c.kw).dx, g.dx)
    assert (mine[dead] == 5).all() and torch.equal(mine[~dead], g.dy[~dead])


def test_module_takes_padded_broadcast_and_strided_inputs():
    """A packed batch with padding behind it, the stream broadcast, the tables of
    different strides: the gradients of the same values laid out plainly."""
    torch.manual_seed(3)
    m = GatedNorm(96, post="rms", pre="layer", device=DEV)
    offsets = torch.tensor([0, 7, 20], dtype=torch.int32, device=DEV)
    x = torch.randn(1, 96, device=DEV, requires_grad=True)
    y = torch.randn(96, 24, device=DEV, requires_grad=True)
    gate = torch.randn(96, device=DEV, requires_grad=True)
    scale = torch.randn(2, 192, device=DEV, requires_grad=True)
    dh, dn = torch.randn(2, 24, 96, device=DEV)
    h, n = m(x.expand(24, 96), y.t(), gate.expand(2, 96), scale[:, ::2], offsets=offsets)
    got = torch.autograd.grad((h, n), (x, y, gate, scale, *m.parameters()), (dh, dn))
    flat = [t.detach().contiguous() for t in (x.expand(24, 96), y.t(), gate.expand(2, 96), scale[:, ::2])]
    want = gated_norm_backward(dh, dn, h.detach(), flat[1], post="rms", post_weight=m.post_weight.detach(),
                               gate=flat[2], weight=m.weight.detach(), bias=m.bias.detach(), scale=flat[3],
                               pre="layer", offsets=offsets)
    assert not h[20:].any() and not n[20:].any()
    # sums of 24 and 2 rows by torch: its own order
    assert torch.allclose(got[0], want.dx.sum(0, keepdim=True), rtol=1e-5, atol=1e-5)
    assert torch.equal(got[1], want.dy.t()) and not got[1][:, 20:].any()
    assert torch.allclose(got[2], want.gate.sum(0), rtol=1e-5, atol=1e-5)
    assert torch.equal(got[3][:, ::2], want.scale) and not got[3][:, 1::2].any()
    for a, b in zip(got[4:], (want.post_weight, want.weight, want.bias)):
        assert torch.equal(a, b)


def test_binding_calls_give_the_layers_results():
    """The wrappers of the C calls, one by one, against fp8.py and norm.py."""
    M, N, K = 40, 130, 200
    w, x, dy = (torch.randn(s, device=DEV) for s in ((N, K), (M, K), (M, N)))
    bias = torch.randn(N, device=DEV)
    layer = Fp8Layer.pack(w, bias)
    q, qt = Fp8Tensor.empty(M, K, DEV), Fp8Tensor.empty(K, M, DEV)
    B.asp_fp8_quantize(x, B.ASP_F32, M, K, K, q.codes, q.scales)
    B.asp_fp8_quantize_t(x, B.ASP_F32, M, K, K, qt.codes, qt.scales)
    for got, want in ((q, quantize(x)), (qt, quantize(x, transpose=True))):
        assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
    a, b = Fp8Tensor.empty(N, K, DEV), Fp8Tensor.empty(K, N, DEV)
    B.asp_fp8_quantize_weight(w, B.ASP_F32, N, K, K, a.codes, a.scales, b.codes, b.scales)
    assert torch.equal(a.codes, layer.codes) and torch.equal(b.codes, layer.codes_t)
    v = torch.empty_like(x)
    B.asp_fp8_dequantize(q.codes, q.scales, M, K, v, B.ASP_F32)
    assert torch.equal(v, q.dequantize())
    want, y, z = layer.forward(x), *(torch.empty((M, N), device=DEV) for _ in range(2))
    ws = layer.workspace(M)
    B.asp_fp8_gemm(q.codes, q.scales, a.codes, a.scales, M, N, K, bias, y, B.ASP_F32)
    B.asp_fp8_forward(x, B.ASP_F32, K, M, N, K, a.codes, a.scales, bias, z, B.ASP_F32, ws, ws.numel())
    assert torch.equal(y, want) and torch.equal(z, want)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(bias)
    ws = layer.workspace(M, backward=True)
    B.asp_fp8_backward(dy, B.ASP_F32, N, x, B.ASP_F32, K, M, N, K, b.codes, b.scales, dx, B.ASP_F32,
                       dw, B.ASP_F32, db, ws, ws.numel())
    assert all(torch.equal(s, t) for s, t in zip((dx, dw, db), layer.backward(dy, x)))

    c = Case(M, K, "f32", "rms", "layer", True, [3, 20, 33])
    h, n = gated_norm(c.x, c.y, **c.kw)
    g = gated_norm_backward(c.dh, c.dn, h, c.y, **c.kw)
    k = c.kw
    h2, n2, dx2, dy2 = (torch.full_like(h, 9.0) for _ in range(4))
    ldt = k["gate"].stride(0)
    B.asp_norm_gate(c.x, c.x.stride(0), c.y, c.y.stride(0), B.ASP_F32, M, K, k["alpha"], B.ASP_NORM_RMS,
                    k["post_weight"], k["gate"], B.ASP_NORM_LAYER, k["weight"], k["bias"], k["scale"],
                    k["shift"], ldt, 2, k["offsets"], EPS, h2, K, n2, B.ASP_F32, K, zero=3)
    assert torch.equal(h2, h) and torch.equal(n2, n)
    made = [torch.full((2, K) if i in (1, 4, 5) else (K,), 9.0, device=DEV) for i in range(6)]
    ws = torch.empty(B.asp_norm_gate_backward_workspace_bytes(M, K, 2), dtype=torch.uint8, device=DEV)
    B.asp_norm_gate_backward(c.dh, c.dh.stride(0), c.dn, c.dn.stride(0), B.ASP_F32, h, K, c.y,
                             c.y.stride(0), B.ASP_F32, M, K, k["alpha"], B.ASP_NORM_RMS, k["post_weight"],
                             k["gate"], B.ASP_NORM_LAYER, k["weight"], k["bias"], k["scale"], ldt, 2,
                             k["offsets"], EPS, dx2, K, dy2, K, 3, *made, K, ws, ws.numel())
    assert all(torch.equal(s, t) for s, t in zip((dx2, dy2, *made), g))


def test_offsets_past_32_bits():
    """The far rows of a large call and the same rows alone: the same bits."""
    M, C = 140_000, 16_384
    x, y = (torch.randn((M, C), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    w = torch.rand(C, device=DEV) + 0.5
    kw = dict(post="rms", post_weight=w, pre="layer", weight=w)
    h, n = gated_norm(x, y, **kw)
    far = slice(M - 50, M)
    for a, b in zip((h, n), gated_norm(x[far].contiguous(), y[far].contiguous(), **kw)):
        assert torch.equal(a[far], b)
    g = gated_norm_backward(x, n, h, y, **kw)
    s = gated_norm_backward(*(t[far].contiguous() for t in (x, n, h, y)), **kw)
    assert torch.equal(g.dx[far], s.dx) and torch.equal(g.dy[far], s.dy)
    del g, s
    _, q = gated_norm(x, y, out="fp8", **kw)
    far = slice(M - 300, M)
    assert torch.equal(q.codes[far], gated_norm(x[far].contiguous(), y[far].contiguous(), out="fp8", **kw)[1].codes)


def test_module_without_a_pre_norm_and_under_capture():
    m = GatedNorm(200, post="layer", pre="none", alpha=0.5, device=DEV)
    x, y = (torch.randn((2, 30, 200), device=DEV, requires_grad=True) for _ in range(2))
    h, n = m(x, y)
    assert n is None
    dh = torch.randn_like(h)
    got = torch.autograd.grad(h, (x, y, m.post_weight), dh)
    want = gated_norm_backward(dh.view(60, 200), None, h.detach().view(60, 200), y.detach().view(60, 200),
                               alpha=0.5, post="layer", post_weight=m.post_weight.detach(), pre="none")
    assert torch.equal(got[0].view(60, 200), want.dx) and torch.equal(got[1].view(60, 200), want.dy)
    assert torch.equal(got[2], want.post_weight)
    with pytest.raises(RuntimeError, match="capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            m(x, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.no_grad(), torch.cuda.graph(graph):
        k = m(x, y)[0]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(k, h)


def test_modules_of_a_bf16_model():
    """Parameters and tables in bf16 are used as their float32 values; gradients come back in
    their types."""
    from wam_asp_w4a4_amd.linear import Fp8Linear
    norm = GatedNorm(96, pre="layer", device=DEV).bfloat16()
    lin = Fp8Linear.from_linear(torch.nn.Linear(96, 70).to(DEV), trainable=True).bfloat16()
    x = torch.randn((20, 96), dtype=torch.bfloat16, device=DEV)
    tab = torch.randn((1, 192), dtype=torch.bfloat16, device=DEV, requires_grad=True)
    scale, shift = tab.chunk(2, dim=1)
    h, n = norm(x, scale=scale, shift=shift)
    z = lin(n)
    want = gated_norm(x, pre="layer", weight=norm.weight.detach().float(), bias=norm.bias.detach().float(),
                      scale=scale.detach().float(), shift=shift.detach().float())[1]
    assert torch.equal(n, want) and z.dtype == torch.bfloat16
    layer = Fp8Layer.pack(lin.weight.detach(), lin.bias.detach().float())
    assert torch.equal(z, layer.forward(want))
    dz = torch.randn_like(z)
    z.backward(dz)
    dn, dw, db = layer.backward(dz, want, dw_dtype="bf16")
    assert torch.equal(lin.weight.grad, dw) and torch.equal(lin.bias.grad, db.bfloat16())
    g = gated_norm_backward(torch.zeros_like(x), dn, h.detach(), pre="layer", weight=norm.weight.detach().float(),
                            bias=norm.bias.detach().float(), scale=scale.detach().float(),
                            shift=shift.detach().float())
    assert torch.equal(tab.grad, torch.cat((g.scale, g.shift), dim=1).bfloat16())
    assert torch.equal(norm.weight.grad, g.weight.bfloat16())


@pytest.mark.parametrize("M,C,dtype,post,pre,offsets", [(40, 1000, "bf16", "rms", "layer", SEQ), (33, 7, "f32", "layer", "rms", None),
                                                        (30, 9001, "bf16", "layer", "layer", SEQ), (700, 1100, "f32", "none", "rms", SEQ),
                                                        (40, 328, "bf16", "rms", "none", [2, 8, 20])])
def test_each_gradient_alone_has_the_same_bits(M, C, dtype, post, pre, offsets):
    print(f"alone {M}x{C} {dtype} {post} {pre}", flush=True)
    c = Case(M, C, dtype, post, pre, True, offsets)
    dn = c.dn if pre != "none" else None
    full = gated_norm_backward(c.dh, dn, c.x, c.y, **c.kw)
    given = [name for name, t in full._asdict().items() if t is not None]
    for need in [[name] for name in given] + [["dx", "gate"], ["dx", "dy"], given[2:], given]:
        got = gated_norm_backward(c.dh, dn, c.x, c.y, need=need, **c.kw)._asdict()
        assert [k for k, v in got.items() if v is not None] == sorted(need, key=given.index)
        assert all(torch.equal(got[k], getattr(full, k)) for k in need), need
    mine = torch.full_like(c.x, 5.0)
    live = torch.from_numpy(c.live).to(DEV)
    assert gated_norm_backward(c.dh, dn, c.x, c.y, dy=mine, need=["dy"], **c.kw).dx is None
    assert torch.equal(mine[live], full.dy[live]) and (mine[~live] == 5).all()


@pytest.mark.parametrize("offsets", [None, [1, 9, 9, 30]])
def test_module_with_frozen_weights_or_an_unused_result(offsets):
    """The gradients are those of the whole call, of a loss in which the unused result has
    the weight 0."""
    c = Case(40, 200, "bf16", "rms", "layer", True, offsets)
    m = GatedNorm(200, post="rms", pre="layer", alpha=0.7, device=DEV)
    tables = {k: c.kw[k].clone() for k in ("gate", "scale", "shift")}
    leaves = [c.x.clone(), c.y.clone(), *tables.values(), *m.parameters()]
    for t in leaves:
        t.requires_grad_()
    x, y, *_ = leaves
    run = lambda: m(x, y, offsets=c.kw["offsets"], **tables)
    for weights in ((1.0, 0.0), (0.0, 1.0)):
        h, n = run()
        want = torch.autograd.grad((h, n), leaves, (c.dh * weights[0], c.dn * weights[1]))
        h, n = run()
        out, d = (h, c.dh) if weights[0] else (n, c.dn)
        got = torch.autograd.grad(out, leaves, d)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    h, n = run()
    want = torch.autograd.grad((h, n), leaves, (c.dh, c.dn))
    m.requires_grad_(False)
    for k in range(1, 5):
        kept = leaves[:k]
        for i, t in enumerate(leaves[:5]):
            t.requires_grad_(i < k)
        h, n = run()
        got = torch.autograd.grad((h, n), kept, (c.dh, c.dn))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("pre", ["rms", "layer", "none"])
@pytest.mark.parametrize("with_y", [False, True])
@pytest.mark.parametrize("offsets", [None, [2, 9, 9, 30]])
def test_module_gives_the_same_with_and_without_gradients(offsets, with_y, pre):
    """The rows of no sequence too: zeros, where offsets are given."""
    c = Case(40, 200, "bf16", "none", pre, False, offsets, affine=False)
    m = GatedNorm(200, pre=pre, device=DEV)
    c.x.requires_grad_()
    kw = dict(y=c.y if with_y else None, offsets=c.kw["offsets"])
    train = m(c.x, **kw)
    assert train[0].requires_grad
    with torch.no_grad():
        plain = m(c.x, **kw)
    for a, b in zip(train, plain):
        assert (a is None) == (b is None)
        assert a is None or torch.equal(a, b) and not b[torch.from_numpy(~c.live).to(DEV)].any()


@pytest.mark.parametrize("M,C", [(5, 7), (33, 1000), (40, 1001), (30, 5001), (30, 9001)])
def test_backward_of_a_bf16_stream_with_a_float32_result(M, C):
    """gated_norm(bf16, out='f32') and its backward: dn in float32 beside bf16 rows."""
    print(f"bf16 stream, float32 dn {M}x{C}", flush=True)
    for post, pre, ld in (("layer", "rms", 0), ("rms", "layer", 3)):
        c = Case(M, C, "bf16", post, pre, True, SEQ if M >= 30 else None, ld=ld)
        h, n = gated_norm(c.x, c.y, out="f32", **c.kw)
        c.check_forward(h, n)
        c.dn = torch.randn((M, C + 5), device=DEV)[:, :C]
        check_backward(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,C", [(3, 129), (33, 1001), (30, 8300), (30, 16384)])
def test_eight_bit_result_of_either_stream_and_of_wide_rows(M, C, dtype):
    print(f"eight bit {M}x{C} {dtype}", flush=True)
    c = Case(M, C, dtype, "rms", "rms", True, SEQ if M >= 30 else None)
    _, n = gated_norm(c.x, c.y, out="f32", **c.kw)
    _, q = gated_norm(c.x, c.y, out="fp8", **c.kw)
    live = torch.from_numpy(c.live).to(DEV)
    codes, s = OF.quantize(host(n))
    np.testing.assert_array_equal(q.codes[live].cpu().numpy(), codes[c.live])
    np.testing.assert_array_equal(q.scales[:, live].cpu().numpy(), OF.layout_scales(s)[:, c.live])


@pytest.mark.parametrize("C", [64, 8192])
def test_the_most_sequences(C):
    """65535 of them, most of one row: the gradients of a few of them alone."""
    G, M = 65535, 66000
    print(f"many sequences {M}x{C}", flush=True)
    torch.manual_seed(C)
    size = torch.ones(G, dtype=torch.int64)
    size[::2000], size[1::2000] = 12, 0
    offsets = torch.cat([torch.tensor([3]), 3 + size.cumsum(0)]).clamp(max=M).to(torch.int32)
    x, y, dh, dn = (torch.randn((M, C), dtype=torch.bfloat16, device=DEV) for _ in range(4))
    table = torch.randn((G, 3, C), device=DEV) * 0.5
    w = 1 + 0.2 * torch.randn(C, device=DEV)
    kw = dict(post="rms", pre="layer", post_weight=w, weight=w, bias=w)
    tables = dict(gate=table[:, 0], scale=table[:, 1], shift=table[:, 2])
    at = offsets.to(DEV)
    h, n = gated_norm(x, y, offsets=at, **tables, **kw)
    g = gated_norm_backward(dh, dn, h, y, offsets=at, **tables, **kw)
    for k in (0, 1, 2, 1999, 2000, 40000, 40001, G - 2, G - 1):
        a, b = offsets[k].item(), offsets[k + 1].item()
        one = {name: t[k:k + 1] for name, t in tables.items()}
        if a == b:
            assert not g.gate[k].any() and not g.scale[k].any() and not g.shift[k].any()
            continue
        part = slice(a, b)
        want = gated_norm(x[part], y[part], **one, **kw)
        assert torch.equal(h[part], want[0]) and torch.equal(n[part], want[1])
        want = gated_norm_backward(dh[part], dn[part], h[part], y[part], **one, **kw)
        assert torch.equal(g.dx[part], want.dx) and torch.equal(g.dy[part], want.dy)
        for name in tables:   # up to 12 terms below 50 in two orders: 2 * 12 * U * 600 < 1e-3
            assert torch.allclose(getattr(g, name)[k], getattr(want, name)[0], rtol=0, atol=1e-3), (name, k)
    live = slice(offsets[0].item(), offsets[-1].item())
    rows = torch.repeat_interleave(torch.arange(G), offsets.diff()).to(DEV)
    m = torch.zeros(C, dtype=torch.float64, device=DEV)
    mass = torch.zeros(C, dtype=torch.float64, device=DEV)
    for i in range(0, rows.numel(), 8192):
        r = slice(i, min(i + 8192, rows.numel()))
        t = dn[live][r].double() * (1 + table[rows[r], 1].double())
        m += t.sum(0)
        mass += t.abs().sum(0)
    # d bias = the sum of dn (1 + scale): each of the rows' and sequences' additions is off by at most U
    assert ((g.bias.double() - m).abs() <= (M + G) * U * mass).all()
