"""The norms after one transformer block and before the next, fused with the
block's gate and the residual scale:

    h = alpha x + gate[g] * post(y)
    n = (pre(h) * weight + bias) * (1 + scale[g]) + shift[g]

``gated_norm`` computes both in one pass (``include/asp.h``, ``asp_norm_gate``,
has the definition); n may leave in the 8-bit format, ready for
``fp8.Fp8Layer.forward``.  ``gated_norm_backward`` gives the gradients of all its
inputs, and ``GatedNorm`` is both as a module.  All arithmetic happens inside
libasp.
"""

from __future__ import annotations

from typing import NamedTuple

import torch

from . import binding as B
from .fp8 import _CODES, Fp8Tensor, _check_rows, _check_vector, _float32, _no_capture, \
    _no_forward_mode, _row_major
from .layer import _Y_DTYPES, _check_ws, _lend, _made_for, _new

KINDS = {"none": B.ASP_NORM_NONE, "rms": B.ASP_NORM_RMS, "layer": B.ASP_NORM_LAYER}


class NormGrads(NamedTuple):
    """Gradients of gated_norm's inputs (None: not given, or not wanted)."""
    dx: torch.Tensor | None
    dy: torch.Tensor | None
    post_weight: torch.Tensor | None
    gate: torch.Tensor | None
    weight: torch.Tensor | None
    bias: torch.Tensor | None
    scale: torch.Tensor | None
    shift: torch.Tensor | None


def _spec(C, device, has_y, post, post_weight, gate, pre, weight, bias, scale, shift, offsets):
    """Checks what x, y share and the tables; (post, pre, G, table row stride)."""
    if post not in KINDS or pre not in KINDS:
        raise ValueError(f"post and pre must be among {sorted(KINDS)}, not {post!r}, {pre!r}")
    if not has_y and (post != "none" or gate is not None):
        raise ValueError("a post norm or gate needs y")
    if pre == "none" and not (weight is bias is scale is shift is None):
        raise ValueError("weight, bias, scale and shift need a pre norm")
    if post == "none" and post_weight is not None:
        raise ValueError("post_weight needs a post norm")
    if post_weight is not None:
        _check_vector(post_weight, "post_weight", C, device)
    if weight is not None:
        _check_vector(weight, "weight", C, device)
    if bias is not None:
        _check_vector(bias, "bias", C, device)
    G = 1
    if offsets is not None:
        if not isinstance(offsets, torch.Tensor) or offsets.dtype != torch.int32:
            raise TypeError("offsets must be an int32 tensor")
        if offsets.dim() != 1 or offsets.numel() < 2 or offsets.device != device \
                or not offsets.is_contiguous():
            raise ValueError(f"offsets must be G + 1 >= 2 contiguous entries on {device}")
        G = offsets.numel() - 1
    ldt = None
    for t, name in ((gate, "gate"), (scale, "scale"), (shift, "shift")):
        if t is None:
            continue
        if isinstance(t, torch.Tensor) and t.dtype is torch.float32 and G == 1 \
                and t.numel() == C == t.shape[-1] and t.dim() <= 2 and t.is_contiguous() \
                and t.device == device and ldt in (None, C):
            ldt = C
            continue
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32:
            raise TypeError(f"{name} must be a float32 tensor")
        if t.shape != (G, C) and not (G == 1 and t.shape == (C,)):
            raise ValueError(f"{name} must be ({G}, {C}), got {tuple(t.shape)}")
        if t.device != device or (C > 1 and t.stride(-1) != 1):
            raise ValueError(f"the rows of {name} must be contiguous and on {device}")
        ld = t.stride(0) if G > 1 else C
        if ldt not in (None, ld) or ld < C:
            raise ValueError("gate, scale and shift must have one row stride, of at least a row")
        ldt = ld
    return KINDS[post], KINDS[pre], G, C if ldt is None else ldt


def gated_norm(x, y=None, *, alpha=1.0, post="none", post_weight=None, gate=None, pre="rms",
               weight=None, bias=None, scale=None, shift=None, offsets=None, eps=1e-6, out=None,
               h=None, n=None, stream=None):
    """(h, n) for the stream x and the block's output y (both M x C, float32 or bf16).

    post, pre: 'none', 'rms' or 'layer' (pre 'none': n is None).  post_weight, weight,
    bias: C float32.  gate, scale, shift: (G, C) float32 (C for one sequence).
    offsets: G + 1 int32, the packed sequences' first rows and the end of the last;
    rows of no sequence are left as they are in h and n where given, and are zeros in
    tensors made here.  out: 'f32', 'bf16' (None: x's type)
    or 'fp8' for an ``Fp8Tensor``.  h, n: tensors to write (h may be x or y); without
    y and with alpha 1, h is x itself and not written unless given.  stream: as in
    ``fp8``, for which everything given must be ready."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a 2-D torch tensor")
    M, C = x.shape
    dev = x.device
    ldx, ldy, same = _check_rows(x, "x", M, C, dev), C, (x.dtype,)
    if y is not None:
        ldy = _check_rows(y, "y", M, C, dev, same)
    post, pre, G, ldt = _spec(C, dev, y is not None, post, post_weight, gate, pre, weight, bias,
                              scale, shift, offsets)
    made, zero = [], 0   # bits of the outputs made here: h, n
    write, ldh = h, C
    if h is not None:
        ldh = _check_rows(h, "h", M, C, dev, same)
    elif y is None and alpha == 1.0 and pre:
        h = x
    else:
        write = h = _new(stream, dev, (M, C), x.dtype)
        made.append(h)
        zero = 1
    scales = None
    if not pre:
        if n is not None or out is not None:
            raise ValueError("out and n need a pre norm")
        values, code, ldn = None, B.ASP_F32, C
    elif out == "fp8" or isinstance(n, Fp8Tensor):
        if out not in (None, "fp8"):
            raise ValueError(f"out {out!r} with an Fp8Tensor n")
        if n is None:
            with _made_for(stream, dev):
                n = Fp8Tensor.empty(M, C, dev)
            made += [n.codes, n.scales]
            zero |= 2
        else:
            if not isinstance(n, Fp8Tensor):
                raise TypeError("out 'fp8' needs an Fp8Tensor n")
            n.check("n")
            if (n.rows, n.cols) != (M, C) or n.codes.device != dev:
                raise ValueError(f"n must be ({M}, {C}) on {dev}")
        values, scales, code, ldn = n.codes, n.scales, B.ASP_E4M3, C
    else:
        if out is not None and out not in _Y_DTYPES:
            raise ValueError(f"out must be 'f32', 'bf16' or 'fp8', not {out!r}")
        ldn = C
        if n is None:
            n = _new(stream, dev, (M, C), x.dtype if out is None else _Y_DTYPES[out])
            made.append(n)
            zero |= 2
        else:
            ldn = _check_rows(n, "n", M, C, dev, _CODES if out is None else (_Y_DTYPES[out],))
        values, code = n, _CODES[n.dtype]
    at = B._at
    B.launch(dev, B.lib().asp_norm_gate, x.data_ptr(), ldx, at(y), ldy, _CODES[x.dtype], M, C, alpha,
             post, at(post_weight), at(gate), pre, at(weight), at(bias), at(scale), at(shift), ldt, G,
             at(offsets), eps, at(write), ldh, at(values), code, ldn, at(scales), zero,
             B.stream_on(stream, dev))
    _lend(stream, *made)
    return h, n


def gated_norm_backward(dh, dn, h, y=None, *, alpha=1.0, post="none", post_weight=None, gate=None,
                        pre="rms", weight=None, bias=None, scale=None, shift=None, offsets=None,
                        eps=1e-6, dx=None, dy=None, need=None, workspace=None, stream=None):
    """Gradients of ``gated_norm`` from dh (of h as it goes on; None: zeros) and dn (of
    n, float32 or bf16; None without a pre norm).  h: the forward's; the options are
    the forward's.  dx, dy: tensors to write (rows of no sequence are left as they
    are; they are zeros in tensors made here).  need: the names of the wanted gradients
    (fields of ``NormGrads``; None: of every given input); the others are not computed, and
    dx and dy alone need no workspace.  A gradient has its input's shape (float32 but for dx
    and dy, which have the stream's type)."""
    if not isinstance(h, torch.Tensor) or h.dim() != 2:
        raise ValueError("h must be a 2-D torch tensor")
    M, C = h.shape
    dev = h.device
    ldh, ldy, lddh, lddn, lddx, lddy = _check_rows(h, "h", M, C, dev), C, C, C, C, C
    same = (h.dtype,)
    if y is not None:
        ldy = _check_rows(y, "y", M, C, dev, same)
    if dh is not None:
        lddh = _check_rows(dh, "dh", M, C, dev, same)
    kpost, kpre, G, ldt = _spec(C, dev, y is not None, post, post_weight, gate, pre, weight, bias,
                                scale, shift, offsets)
    if (dn is not None) != bool(kpre):
        raise ValueError("dn belongs to the pre norm's result")
    if dn is not None:
        lddn = _check_rows(dn, "dn", M, C, dev)
    if dh is None and dn is None:
        raise ValueError("neither dh nor dn is given")
    if y is None and dy is not None:
        raise ValueError("dy without y")
    # the inputs whose gradients are wanted
    wanted = NormGrads(h, y, post_weight, gate, weight, bias, scale, shift)
    if need is not None:
        need = tuple(need)
        for name in need:
            if name not in NormGrads._fields or getattr(wanted, name) is None:
                raise ValueError(f"need names {name!r}: no gradient of a given input")
        if dx is not None and "dx" not in need or dy is not None and "dy" not in need:
            raise ValueError("a tensor for a gradient that need does not name")
        if not need:
            return NormGrads(*8 * (None,))
        wanted = NormGrads(*(t if name in need else None for name, t in wanted._asdict().items()))
    made, zero = [], 0   # bits of the outputs made here: dx, dy

    def new(shape, dtype=torch.float32):
        made.append(_new(stream, dev, shape, dtype))
        return made[-1]

    def like(*inputs):
        # one allocation for those of one shape
        given = [t for t in inputs if t is not None]
        if any(t.shape != given[0].shape for t in given):
            return [None if t is None else new(t.shape) for t in inputs]
        rows = iter(new((len(given), *given[0].shape)).unbind(0) if given else ())
        return [None if t is None else next(rows) for t in inputs]

    if dx is not None:
        lddx = _check_rows(dx, "dx", M, C, dev, same)
    elif wanted.dx is not None:
        dx = new((M, C), h.dtype)
        zero = 1
    if dy is not None:
        lddy = _check_rows(dy, "dy", M, C, dev, same)
    elif wanted.dy is not None:
        dy = new((M, C), h.dtype)
        zero |= 2
    d_post_weight, d_weight, d_bias = like(wanted.post_weight, wanted.weight, wanted.bias)
    d_gate, d_scale, d_shift = like(wanted.gate, wanted.scale, wanted.shift)
    size = 0
    if not (d_post_weight is d_weight is d_bias is d_gate is d_scale is d_shift is None):
        size = B.asp_norm_gate_backward_workspace_bytes(M, C, G)
        if workspace is None:
            workspace = _new(stream, dev, size, torch.uint8)
    if workspace is not None:
        _check_ws(workspace, size, dev)
    at = B._at
    B.launch(dev, B.lib().asp_norm_gate_backward, at(dh), lddh, at(dn), lddn,
             B.ASP_F32 if dn is None else _CODES[dn.dtype], h.data_ptr(), ldh, at(y), ldy,
             _CODES[h.dtype], M, C, alpha, kpost, at(post_weight), at(gate), kpre, at(weight),
             at(bias), at(scale), ldt, G, at(offsets), eps, at(dx), lddx, at(dy), lddy, zero,
             at(d_post_weight), at(d_gate), at(d_weight), at(d_bias), at(d_scale), at(d_shift), C,
             at(workspace), 0 if workspace is None else workspace.numel(), B.stream_on(stream, dev))
    _lend(stream, *made)
    return NormGrads(dx, dy, d_post_weight, d_gate, d_weight, d_bias, d_scale, d_shift)


def _module_norm(x, y, offsets, h=None, **options):
    """``gated_norm`` with zeros in h's rows of no sequence also where h would be x itself."""
    if y is None and options["alpha"] == 1.0 and offsets is not None:
        h = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
    return gated_norm(x, y, h=h, offsets=offsets, **options)


class _GatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, post_weight, gate, weight, bias, scale, shift, offsets, options):
        ctx.set_materialize_grads(False)
        given = dict(post_weight=post_weight, gate=gate, weight=weight, bias=bias, scale=scale,
                     shift=shift)
        h = None
        if y is None and options["alpha"] == 1.0 and offsets is None:
            # written all the same: a stream returned as it came would share its version
            h = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        h, n = _module_norm(x, y, h=h, offsets=offsets, **given, **options)
        ctx.save_for_backward(h, y, *given.values(), offsets)
        ctx.options = options
        return h, n

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh, dn):
        _no_capture()
        h, y, *tensors, offsets = ctx.saved_tensors
        given = dict(zip(NormGrads._fields[2:], tensors))
        need = [name for name, n in zip(NormGrads._fields, ctx.needs_input_grad) if n]
        options = ctx.options
        if dh is None and dn is None or not need:
            return 10 * (None,)
        zeros = {}
        if dn is None and options["pre"] != "none":
            # n is not used: h alone goes on, and what only n reads has zero gradients
            options = {**options, "pre": "none"}
            for name in ("weight", "bias", "scale", "shift"):
                t = given.pop(name)
                if name in need:
                    zeros[name] = torch.zeros_like(t)
            need = [name for name in need if name not in zeros]
        g = gated_norm_backward(None if dh is None else dh.contiguous(),
                                None if dn is None else dn.contiguous(), h, y, need=need,
                                offsets=offsets, **given, **options)
        return (*g._replace(**zeros), None, None)


class GatedNorm(torch.nn.Module):
    """``gated_norm`` with its weights as parameters, differentiable in every input.

    x, y: (..., C) of one shape, or either as its rows (M, C); gate, scale, shift: (G, C) or
    (C), taken as float32 like the weights; returns (h, n) of x's shape (n None for pre
    'none'; rows of no sequence are zeros; without gradients, offsets, y and a factor alpha,
    h is x itself).  Gradients are reverse mode; forward-mode tangents are refused.  Under a HIP
    graph capture, gradients are refused: capture ``gated_norm`` and
    ``gated_norm_backward``, which keep no graph of their own."""

    def __init__(self, channels, post="none", pre="rms", alpha=1.0, eps=1e-6, device=None):
        super().__init__()
        if post not in KINDS or pre not in KINDS:
            raise ValueError(f"post and pre must be among {sorted(KINDS)}, not {post!r}, {pre!r}")
        self.channels, self.post, self.pre, self.alpha, self.eps = channels, post, pre, alpha, eps

        def parameter(used, value):
            return torch.nn.Parameter(torch.full((channels,), value, device=device)) if used else None

        self.post_weight = parameter(post != "none", 1.0)
        self.weight = parameter(pre != "none", 1.0)
        self.bias = parameter(pre == "layer", 0.0)

    def forward(self, x, y=None, gate=None, scale=None, shift=None, offsets=None):
        if x.shape[-1] != self.channels:
            raise ValueError(f"x has {x.shape[-1]} channels, the norm {self.channels}")
        if y is None and self.post != "none":
            raise ValueError("a post norm needs y")
        if y is not None and y.shape != x.shape and not (
                2 in (x.dim(), y.dim()) and y.shape[-1] == self.channels
                and y.numel() == x.numel()):
            raise ValueError(f"y must have the shape of x or of its rows, {tuple(x.shape)}, "
                             f"got {tuple(y.shape)}")
        flat = [None if t is None else _row_major(t.reshape(-1, self.channels)) for t in (x, y)]
        post_weight, weight, bias, gate, scale, shift = map(
            _float32, (self.post_weight, self.weight, self.bias, gate, scale, shift))
        tables = [t for t in (gate, scale, shift) if t is not None]
        if len({(t.dim(), t.stride()) for t in tables}) > 1 or any(_row_major(t) is not t for t in tables):
            gate, scale, shift = (None if t is None else t.contiguous() for t in (gate, scale, shift))
        options = dict(post=self.post, pre=self.pre, alpha=self.alpha, eps=self.eps)
        tensors = (post_weight, gate, weight, bias, scale, shift)
        _no_forward_mode(*flat, *tensors)
        if torch.is_grad_enabled() and any(t is not None and t.requires_grad
                                           for t in (*flat, *tensors)):
            _no_capture()
            h, n = _GatedNorm.apply(*flat, *tensors, offsets, options)
        else:
            names = ("post_weight", "gate", "weight", "bias", "scale", "shift")
            h, n = _module_norm(*flat, offsets, **dict(zip(names, tensors)), **options)
        return h.reshape(x.shape), None if n is None else n.reshape(x.shape)

    def extra_repr(self) -> str:
        return (f"{self.channels}, post={self.post!r}, pre={self.pre!r}, alpha={self.alpha}, "
                f"eps={self.eps}")
