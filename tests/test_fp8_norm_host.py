"""Refusals of the 8-bit layer and the gated norms (CPU: nothing here reaches a
kernel; pointers that reach the C ABI are fake and rejected before any use), and
the modules that hold them."""

import ctypes

import pytest
import torch
import torch.autograd.forward_ad as forward_ad

from wam_asp_w4a4_amd import binding as B
from wam_asp_w4a4_amd import fp8, norm
from wam_asp_w4a4_amd.linear import ASPLinear, Fp8Linear, InstallError, install

FAKE = 0x7F0000000000


def layer(N=64, K=200, bias=True, backward=True):
    q, t = fp8.Fp8Tensor.empty(N, K, "cpu"), fp8.Fp8Tensor.empty(K, N, "cpu")
    return fp8.Fp8Layer(N, K, q.codes, q.scales, t.codes if backward else None,
                        t.scales if backward else None, torch.zeros(N) if bias else None)


def test_sizes():
    assert B.asp_fp8_sizes(3, 130) == (3 * 256, 3 * 4)
    assert B.asp_fp8_sizes(5, 513) == (5 * 640, 2 * 5 * 4)
    assert B.asp_fp8_sizes(0, 1) == (0, 0)
    assert B.asp_fp8_workspace_bytes(16, 4096, 4096) == 0       # one kernel, nothing kept
    assert B.asp_fp8_workspace_bytes(17, 64, 128) >= 17 * 128 + 17 * 4
    for rows, cols in ((-1, 4), (4, 0), (4, (1 << 20) + 1), (1 << 31, 4)):
        with pytest.raises(B.ASPError) as ei:
            B.asp_fp8_sizes(rows, cols)
        assert ei.value.status == 2


@pytest.mark.parametrize("M,N,K", [(4, 0, 128), (4, (1 << 30) + 1, 128), (-1, 4, 128), (4, 4, 0)])
def test_shapes_are_refused_everywhere(M, N, K):
    for call in (lambda: B.asp_fp8_workspace_bytes(M, N, K),
                 lambda: B.asp_fp8_gemm_workspace_bytes(M, N, K),
                 lambda: B.asp_fp8_backward_workspace_bytes(M, N, K),
                 lambda: B.asp_fp8_gemm(None, None, None, None, M, N, K, None, None, 0)):
        with pytest.raises(B.ASPError) as ei:
            call()
        assert ei.value.status == 2
    with pytest.raises(B.ASPError) as ei:      # the backward contracts over M and N
        B.asp_fp8_backward_workspace_bytes((1 << 20) + 1, 4, 4)
    assert ei.value.status == 2


def _status(fn, *args):
    return getattr(B.lib(), fn)(*args)


def test_c_calls_validate_before_any_launch():
    q = lambda x=FAKE, dt=0, rows=4, cols=100, ld=100, c=FAKE, s=FAKE: _status(
        "asp_fp8_quantize", x, dt, rows, cols, ld, c, s, None)
    assert q(dt=2) == 1 and q(x=None) == 1 and q(c=None) == 1
    assert q(ld=99) == 2 and q(rows=-1) == 2 and q(cols=0) == 2
    assert q(x=FAKE + 2) == 3 and q(c=FAKE + 8) == 3 and q(s=FAKE + 4) == 3
    assert q(rows=0, x=None, c=None, s=None) == 0
    assert q(rows=1 << 27, cols=4096, ld=4096) == 2        # 2^28 workgroups: no launch takes them
    t = lambda **o: _status("asp_fp8_quantize_t", FAKE, 1, o.get("rows", 4), 100, 100, o.get("c", FAKE), FAKE, None)
    assert t(c=None) == 1 and t(rows=(1 << 20) + 1) == 2 and t(rows=0) == 0
    w = lambda ct=FAKE, st=FAKE, N=4: _status("asp_fp8_quantize_weight", FAKE, 0, N, 100, 100, FAKE, FAKE, ct, st, None)
    assert w(ct=None) == 1 and w(st=None) == 1 and w(N=0) == 2
    need = B.asp_fp8_workspace_bytes(64, 32, 200)
    f = lambda x=FAKE, ldx=200, w=FAKE, y=FAKE, ydt=0, ws=FAKE, nb=need, bias=None, M=64: _status(
        "asp_fp8_forward", x, 1, ldx, M, 32, 200, w, FAKE, bias, y, ydt, ws, nb, None)
    assert f(x=None) == 1 and f(w=None) == 1 and f(y=None) == 1 and f(ws=None) == 1 and f(ydt=2) == 1
    assert f(ldx=199) == 2 and f(x=FAKE + 1) == 3 and f(ws=FAKE + 16) == 3 and f(bias=FAKE + 2) == 3
    assert f(nb=need - 1) == 5 and f(M=0, x=None) == 0
    need = B.asp_fp8_backward_workspace_bytes(64, 32, 200)
    b = lambda dy=FAKE, x=FAKE, wt=FAKE, dx=FAKE, dw=FAKE, db=FAKE, nb=need: _status(
        "asp_fp8_backward", dy, 1, 32, x, 1, 200, 64, 32, 200, wt, FAKE, dx, 1, dw, 0, db, FAKE, nb, None)
    assert b(dy=None) == 1 and b(x=None) == 1 and b(wt=None) == 1 and b(nb=need - 1) == 5
    assert b(dw=FAKE + 2) == 3
    assert b(dx=None, dw=None, db=None) == 0      # nothing is asked for
    # few tiles of a long K: slices, whose sums need a workspace
    need = B.asp_fp8_gemm_workspace_bytes(512, 512, 65536)
    assert need > 0 and B.asp_fp8_gemm_workspace_bytes(64, 64, 8192) == 0
    g = lambda a=FAKE, ws=FAKE, nb=need - 1: _status(
        "asp_fp8_gemm", a, FAKE, FAKE, FAKE, 512, 512, 65536, None, FAKE, 0, ws, nb, None)
    assert g(a=None) == 1 and g(a=FAKE + 4) == 3 and g() == 5 and g(ws=None) == 1


def _norm(**o):
    a = dict(x=FAKE, ldx=96, y=FAKE, ldy=96, dtype=0, M=8, C=96, alpha=1.0, post=1, pw=None, gate=None, pre=1,
             w=None, b=None, sc=None, sh=None, ldt=96, G=1, off=None, eps=1e-6, h=FAKE, ldh=96, n=FAKE, ndt=0,
             ldn=96, ns=None, zero=0)
    a.update(o)
    return _status("asp_norm_gate", *a.values(), None)


def test_norm_refusals():
    assert _norm(x=None) == 1 and _norm(n=None) == 1 and _norm(dtype=2) == 1 and _norm(ndt=3) == 1
    assert _norm(post=3) == 1 and _norm(pre=-1) == 1 and _norm(eps=float("nan")) == 1 and _norm(eps=-1e-6) == 1
    assert _norm(y=None) == 1 and _norm(y=None, post=0, gate=FAKE) == 1 and _norm(post=0, pw=FAKE) == 1
    assert _norm(pre=0) == 1 and _norm(pre=0, n=None, h=None) == 1 and _norm(pre=0, n=None, sc=FAKE) == 1
    assert _norm(G=2) == 1 and _norm(ndt=2) == 1        # no offsets; no scales
    assert _norm(C=0) == 2 and _norm(C=16385) == 2 and _norm(M=-1) == 2 and _norm(ldx=95) == 2
    assert _norm(G=0) == 2 and _norm(G=2, off=FAKE, ldt=95) == 2 and _norm(ldn=95) == 2
    assert _norm(x=FAKE + 2) == 3 and _norm(off=FAKE + 2) == 3 and _norm(w=FAKE + 1) == 3
    assert _norm(ndt=2, n=FAKE + 8, ns=FAKE) == 3
    assert _norm(zero=4) == 1 and _norm(zero=-1) == 1 and _norm(zero=1, h=None) == 1
    assert _norm(M=0, x=None, n=None) == 0
    need = B.asp_norm_gate_backward_workspace_bytes(8, 96, 1)

    def back(**o):
        a = dict(dh=FAKE, lddh=96, dn=FAKE, lddn=96, dndt=0, h=FAKE, ldh=96, y=FAKE, ldy=96, dtype=0, M=8, C=96,
                 alpha=1.0, post=1, pw=None, gate=None, pre=1, w=None, b=None, sc=None, ldt=96, G=1, off=None,
                 eps=1e-6, dx=FAKE, lddx=96, dy=FAKE, lddy=96, zero=0, dpw=None, dg=None, dw=FAKE, db=None, dsc=None,
                 dsh=None, ldd=96, ws=FAKE, nb=need)
        a.update(o)
        return _status("asp_norm_gate_backward", *a.values(), None)

    assert back(dn=None) == 1 and back(h=None) == 1 and back(y=None) == 1 and back(ws=None) == 1
    assert back(pre=0) == 1 and back(pre=0, dn=None, dw=None, dh=None) == 1 and back(post=0, dpw=FAKE) == 1
    assert back(lddn=95) == 2 and back(dx=FAKE + 2) == 3 and back(nb=need - 1) == 5
    assert back(zero=4) == 1 and back(zero=1, dx=None) == 1 and back(zero=2, dy=None) == 1
    assert back(dx=None, dy=None, dw=None) == 0


@pytest.mark.parametrize("case", ["wrong K", "3-D", "fp16", "overlap", "columns", "list", "y shape", "y dtype",
                                  "ws dtype", "ws small", "codes of another size"])
def test_layer_rejects_before_launch(case):
    l, x, kw = layer(), torch.zeros((40, 200)), {}
    if case == "wrong K":
        x = torch.zeros((40, 128))
    elif case == "3-D":
        x = x[None]
    elif case == "fp16":
        x = x.half()
    elif case == "overlap":
        x = torch.zeros(200).expand(40, 200)
    elif case == "columns":
        x = torch.zeros((200, 40)).t()
    elif case == "list":
        x = [[0.0] * 200]
    elif case == "y shape":
        kw["y"] = torch.empty((40, 65))
    elif case == "y dtype":
        kw["y"] = torch.empty((40, 64), dtype=torch.bfloat16)
    elif case == "ws dtype":
        kw["workspace"] = torch.empty(1 << 16)
    elif case == "ws small":
        kw["workspace"] = torch.empty(16, dtype=torch.uint8)
    else:
        x = fp8.Fp8Tensor.empty(40, 300, "cpu")
    with pytest.raises((ValueError, TypeError)):
        l.forward(x, **kw)


def test_layer_pieces_must_fit():
    l = layer()
    with pytest.raises(ValueError):
        fp8.Fp8Layer(l.N, l.K, l.codes, l.scales, l.codes_t, None, None)
    with pytest.raises(ValueError):
        fp8.Fp8Layer(l.N, l.K + 100, l.codes, l.scales, None, None, None)
    with pytest.raises(ValueError):
        fp8.Fp8Layer(l.N, l.K, l.codes, l.scales, None, None, torch.zeros(3))
    with pytest.raises(TypeError):
        fp8.Fp8Layer(l.N, l.K, l.codes.float(), l.scales, None, None, None)
    with pytest.raises(ValueError, match="backward=True"):
        layer(backward=False).backward(torch.zeros((4, 64)))
    with pytest.raises(ValueError):
        l.backward(torch.zeros((4, 64)), torch.zeros((5, 200)))
    assert layer(bias=False).backward(torch.zeros((4, 64)), need_dx=False) == (None, None, None)


@pytest.mark.parametrize("case", ["kind", "gate without y", "post without y", "weight without pre", "gate shape",
                                  "strides", "offsets dtype", "offsets size", "y type", "n fp8", "out name",
                                  "out without pre", "bf16 weight"])
def test_gated_norm_rejects_before_launch(case):
    x = torch.zeros((6, 32))
    y, kw = x.clone(), {}
    off = torch.tensor([0, 3, 6], dtype=torch.int32)
    if case == "kind":
        kw["pre"] = "batch"
    elif case == "gate without y":
        y, kw["gate"] = None, torch.zeros(32)
    elif case == "post without y":
        y, kw["post"] = None, "rms"
    elif case == "weight without pre":
        kw.update(pre="none", weight=torch.zeros(32))
    elif case == "gate shape":
        kw.update(gate=torch.zeros((3, 32)), offsets=off)
    elif case == "strides":
        kw.update(gate=torch.zeros((2, 32)), scale=torch.zeros((2, 64))[:, :32], offsets=off)
    elif case == "offsets dtype":
        kw["offsets"] = off.long()
    elif case == "offsets size":
        kw["offsets"] = off[:1]
    elif case == "y type":
        y = y.bfloat16()
    elif case == "n fp8":
        kw.update(out="fp8", n=torch.zeros((6, 32)))
    elif case == "out name":
        kw["out"] = "f16"
    elif case == "out without pre":
        kw.update(pre="none", out="f32")
    else:
        kw["weight"] = torch.zeros(32, dtype=torch.bfloat16)
    with pytest.raises((ValueError, TypeError)):
        norm.gated_norm(x, y, **kw)


def test_gated_norm_backward_rejects_before_launch():
    x = torch.zeros((6, 32))
    for args, kw in (((None, None, x), dict(pre="none")), ((x, x, x), dict(pre="none")), ((x, None, x), {}),
                     ((x, x, x), dict(dy=x)), ((x.bfloat16(), x, x), {}), ((x, x[:5], x), {})):
        with pytest.raises(ValueError if args[0] is None or args[0].dtype == x.dtype else TypeError):
            norm.gated_norm_backward(*args, **kw)


CPU_CALLS = {
    "quantize": lambda x: fp8.quantize(x),
    "quantize transposed": lambda x: fp8.quantize(x, transpose=True),
    "dequantize": lambda x: fp8.Fp8Tensor.empty(40, 200, "cpu").dequantize(),
    "pack": lambda x: fp8.Fp8Layer.pack(x),
    "forward": lambda x: layer().forward(x),
    "forward of codes": lambda x: layer().forward(fp8.Fp8Tensor.empty(40, 200, "cpu")),
    "backward": lambda x: layer().backward(torch.zeros((40, 64)), x),
    "norm": lambda x: norm.gated_norm(x, x, post="rms"),
    "norm to codes": lambda x: norm.gated_norm(x, out="fp8"),
    "norm backward": lambda x: norm.gated_norm_backward(x, x, x, x, weight=torch.ones(200)),
    "norm module": lambda x: norm.GatedNorm(200)(x),
    "norm module, frozen": lambda x: norm.GatedNorm(200).requires_grad_(False)(x),
    "linear": lambda x: Fp8Linear(layer())(x),
    "linear, trainable": lambda x: Fp8Linear.from_linear(torch.nn.Linear(200, 64), trainable=True)(x),
    "from_linear": lambda x: Fp8Linear.from_linear(torch.nn.Linear(200, 64)),
}


@pytest.mark.parametrize("call", list(CPU_CALLS))
def test_cpu_tensors_never_reach_the_library(call, monkeypatch):
    """Every other argument is right: only the device is not."""
    reached = []
    for name in B.SIGNATURES:
        if name.startswith(("asp_fp8", "asp_norm")) and not name.endswith(("_bytes", "_sizes")):
            monkeypatch.setattr(B.lib(), name, lambda *a, name=name: reached.append(name) or 0)
    with pytest.raises(ValueError, match="GPU"):
        CPU_CALLS[call](torch.zeros((40, 200)))
    assert not reached


def test_install_takes_either_kind():
    m = torch.nn.Sequential(torch.nn.Linear(200, 64), torch.nn.GELU(), torch.nn.Linear(64, 200, bias=False))
    assert install(m, {"0": layer(64, 200), "2": layer(200, 64, bias=False)}) == ["0", "2"]
    assert isinstance(m[0], Fp8Linear) and isinstance(m[2], Fp8Linear) and not isinstance(m[0], ASPLinear)
    assert (m[0].in_features, m[0].out_features) == (200, 64) and m[0].bias is not None
    m = torch.nn.Sequential(torch.nn.Linear(200, 64))
    with pytest.raises(InstallError, match="packed 200 -> 32"):
        install(m, {"0": layer(32, 200)})
    with pytest.raises(ValueError):
        Fp8Linear()
    with pytest.raises(ValueError):
        Fp8Linear(layer(), bias=torch.zeros(64))


@pytest.mark.parametrize("xs,ys,fits", [((4, 96), (8, 48), False), ((4, 96), (96, 4), False), ((4, 96), (384,), False),
                                        ((2, 6, 96), (3, 4, 96), False), ((2, 6, 96), (6, 2, 96), False),
                                        ((4, 96), (1, 96), False), ((2, 6, 96), (2, 1, 96), False),
                                        ((4, 96), (4, 96), True), ((2, 6, 96), (12, 96), True),
                                        ((12, 96), (3, 4, 96), True), ((96,), (1, 96), True)])
def test_module_takes_a_y_of_the_streams_rows_only(xs, ys, fits):
    """What fits gets as far as the refusal of CPU tensors."""
    m = norm.GatedNorm(96, post="rms")
    for frozen in (False, True):
        with pytest.raises(ValueError, match="GPU" if fits else "y must have the shape"):
            m.requires_grad_(not frozen)(torch.zeros(xs), torch.zeros(ys))


@pytest.mark.parametrize("frozen", [False, True])
def test_forward_mode_is_refused(frozen, monkeypatch):
    """The library's calls are replaced: a tangent must not get that far, wherever it rides."""
    monkeypatch.setattr(B, "launch", lambda *a: None)
    m = norm.GatedNorm(200, post="rms", pre="layer").requires_grad_(not frozen)
    packed = Fp8Linear(layer())
    trained = Fp8Linear.from_linear(torch.nn.Linear(200, 64), trainable=True).requires_grad_(not frozen)
    x, table = torch.ones((6, 200)), torch.ones(200)
    with forward_ad.dual_level():
        dx, dt = (forward_ad.make_dual(t, t.clone()) for t in (x, table))
        weight = forward_ad.make_dual(trained.weight.detach(), torch.ones((64, 200)))
        calls = [lambda: m(dx, x), lambda: m(x, dx), lambda: m(x, x, gate=dt), lambda: m(x, x, shift=dt),
                 lambda: packed(dx), lambda: trained(dx),
                 lambda: torch.func.functional_call(m, {"weight": dt}, (x, x)),
                 lambda: torch.func.functional_call(trained, {"weight": weight}, (x,))]
        for i, call in enumerate(calls):
            with pytest.raises(RuntimeError, match="forward-mode"):
                call()
                print("no error:", i)
        for m_, args in ((m, (x, x)), (packed, (x,)), (trained, (x,))):
            m_(*args)                         # none of its tensors has a tangent
    with pytest.raises(RuntimeError, match="forward-mode"):
        torch.func.jvp(packed, (x,), (x,))


def test_a_bias_that_was_converted_is_not_read_as_float32(monkeypatch):
    """A bias parameter follows the module's type; the kernels read float32 of N entries."""
    seen = []

    def launch(device, fn, x, dtype, ld, M, N, K, codes, scales, bias, *rest):
        seen.append((bias, [] if bias is None else list((ctypes.c_float * N).from_address(bias))))

    monkeypatch.setattr(B, "launch", launch)
    l = layer(bias=False)
    l = fp8.Fp8Layer(l.N, l.K, l.codes, l.scales, l.codes_t, l.scales_t, torch.nn.Parameter(torch.arange(64.0)))
    m, x = Fp8Linear(l), torch.zeros((4, 200))
    values = list(range(64))
    m(x)
    assert seen[-1] == (l.bias.data_ptr(), values)
    m.bfloat16()
    assert l.bias.dtype == torch.bfloat16
    with pytest.raises(TypeError, match="bias must be a float32 tensor"):
        l.forward(x)
    for grad in (True, False):                 # the module uses its values
        m.bias.requires_grad_(grad)
        m(x)
        assert seen[-1][1] == values
    m.bias = torch.nn.Parameter(torch.ones(64))     # another one in its place
    m(x)
    assert seen[-1] == (m.bias.data_ptr(), [1.0] * 64)
    m.bias = None
    m(x)
    assert seen[-1][0] is None
    m.bias = torch.nn.Parameter(torch.ones(64, device="meta"))
    with pytest.raises(ValueError, match="bias"):
        m(x)


def test_offsets_changed_before_the_backward_are_noticed(monkeypatch):
    monkeypatch.setattr(B, "launch", lambda *a: None)
    m = norm.GatedNorm(32)
    off = torch.tensor([0, 3, 6], dtype=torch.int32)
    for change in (False, True):
        n = m(torch.zeros((6, 32)), offsets=off)[1]
        if change:
            off[1] = 4                      # the next batch's, in the same buffer
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                n.sum().backward()
        else:
            n.sum().backward()


BACKWARD_ARGS = ("dh lddh dn lddn dn_dtype h ldh y ldy dtype M C alpha post post_weight_in gate_in pre weight_in bias_in "
                 "scale_in ldt G offsets eps dx lddx dy lddy zero post_weight gate weight bias scale shift ldd ws "
                 "ws_bytes stream").split()


@pytest.mark.parametrize("used", ["h and n", "h", "n"])
@pytest.mark.parametrize("trained", [("x",), ("y",), ("x", "y", "weight"), ("gate",), ("y", "shift"), ("post_weight",)])
def test_backward_asks_the_library_for_the_wanted_gradients_only(trained, used, monkeypatch):
    """By the pointers that the call passes: NULL for what nobody wants, and for a result
    that nothing uses."""
    calls = []
    monkeypatch.setattr(B, "launch", lambda device, fn, *args: calls.append(args))
    m = norm.GatedNorm(32, post="rms", pre="layer").requires_grad_(False)
    t = {"x": torch.ones((6, 32)), "y": torch.ones((6, 32)), "gate": torch.ones(32), "scale": torch.ones(32),
         "shift": torch.ones(32)}
    for name in trained:
        (t[name] if name in t else getattr(m, name)).requires_grad_()
    h, n = m(**t)
    wanted = [t[name] if name in t else getattr(m, name) for name in trained]
    loss = {"h and n": (h, n), "h": (h,), "n": (n,)}[used]
    del calls[:]
    got = torch.autograd.grad(loss, wanted, [torch.ones_like(o) for o in loss])
    assert all(g.shape == w.shape for g, w in zip(got, wanted))
    names = {"x": "dx", "y": "dy"}
    n_only = {"weight", "bias", "scale", "shift"}
    asked = {names.get(k, k) for k in trained if used != "h" or k not in n_only}
    for name, g in zip(trained, got):
        assert names.get(name, name) in asked or not g.any()
    if not asked:
        assert not calls
        return
    a = dict(zip(BACKWARD_ARGS, calls[0]))
    assert len(calls) == 1 and len(calls[0]) == len(BACKWARD_ARGS)
    given = {k for k in norm.NormGrads._fields if a[k] is not None}
    assert given == asked
    assert (a["dh"] is None) == (used == "n") and (a["dn"] is None) == (used == "h")
    assert (a["ws"] is None) == (asked <= {"dx", "dy"})
    assert a["zero"] == ("dx" in asked) + 2 * ("dy" in asked)


def test_need_is_checked():
    x, w = torch.zeros((6, 32)), torch.ones(32)
    for kw, why in ((dict(need=["dz"]), "dz"), (dict(need=["dy"]), "dy"), (dict(need=["weight", "gate"], weight=w), "gate"),
                    (dict(need=["weight"], weight=w, dx=x), "does not name"), (dict(dy=x), "dy without y")):
        with pytest.raises(ValueError, match=why):
            norm.gated_norm_backward(x, x, x, **kw)
    assert norm.gated_norm_backward(x, x, x, need=[]) == (None,) * 8
    assert norm.gated_norm_backward(x, x, x, need=iter(())) == (None,) * 8


def test_need_may_be_read_once(monkeypatch):
    monkeypatch.setattr(B, "launch", lambda *a: None)
    x, w = torch.zeros((6, 32)), torch.ones(32)
    g = norm.gated_norm_backward(x, x, x, weight=w, need=(name for name in ("dx", "weight")))
    assert g.dx.shape == x.shape and g.weight.shape == w.shape
    assert norm.gated_norm_backward(x, x, x, weight=w, need={"weight"}).dx is None


@pytest.mark.parametrize("x_type,y_dtype,dx,dw", [(torch.float32, None, 0, 0), (torch.bfloat16, None, 1, 1),
                                                  (torch.float32, "bf16", 0, 1), (torch.bfloat16, "bf16", 1, 1),
                                                  (torch.float32, "f32", 0, 0), (torch.bfloat16, "f32", 0, 0)])
def test_gradients_have_the_bits_of_their_inputs(x_type, y_dtype, dx, dw, monkeypatch):
    """The types that the module's backward asks the library for (0 float32, 1 bf16): a
    gradient of a float32 x is not computed in bf16 because y is."""
    calls = []
    monkeypatch.setattr(B, "launch", lambda device, fn, *args: calls.append(args))
    weight = torch.nn.Parameter(torch.zeros((64, 200), dtype=torch.bfloat16 if dw else torch.float32))
    m = Fp8Linear(weight=weight, y_dtype=y_dtype)
    x = torch.zeros((6, 200), dtype=x_type, requires_grad=True)
    y = m(x)
    assert y.dtype == {"f32": torch.float32, "bf16": torch.bfloat16, None: x_type}[y_dtype]
    y.sum().backward()
    assert calls[-1][12] == dx and calls[-1][14] == dw
    assert x.grad.dtype == x_type and weight.grad.dtype == weight.dtype


def test_result_types_are_checked():
    for call in (lambda: Fp8Linear(layer(), y_dtype="f16"), lambda: layer().forward(torch.zeros((4, 200)), "f16"),
                 lambda: layer().backward(torch.zeros((4, 64)), dx_dtype="f16"),
                 lambda: layer().backward(torch.zeros((4, 64)), torch.zeros((4, 200)), dw_dtype="f16")):
        with pytest.raises(ValueError, match="must be 'f32'"):
            call()
