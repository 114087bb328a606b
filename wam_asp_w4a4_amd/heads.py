"""The norms of a block's queries and keys, each head by itself, with the rotation
by their positions in the same pass:

    u = norm(v) * weight                  over a head's D elements
    y: pairs (a, b) of u turned to (a cos - b sin, a sin + b cos)

``head_norm`` computes it for the queries and keys of T tokens (``include/asp.h``,
``asp_head_norm``, has the definition), ``head_norm_backward`` gives the gradients,
and ``HeadNorm`` is both as a module.  All arithmetic happens inside libasp.
"""

from __future__ import annotations

from typing import NamedTuple

import torch

from . import binding as B
from .fp8 import _CODES, _check_vector, _float32, _no_capture, _no_forward_mode
from .layer import _Y_DTYPES, _check_ws, _lend, _new
from .norm import KINDS

LAYOUTS = {"pairs": B.ASP_ROTATE_PAIRS, "halves": B.ASP_ROTATE_HALVES}


class HeadNormGrads(NamedTuple):
    """Gradients of head_norm's inputs (None: not given, or not wanted)."""
    dq: torch.Tensor | None
    dk: torch.Tensor | None
    q_weight: torch.Tensor | None
    k_weight: torch.Tensor | None


def _check_heads(t, name, shape, device, dtypes=_CODES):
    """t must be (T, H, D) with contiguous heads (None in `shape`: any number).  Returns its
    token and head strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    have = t.shape
    if len(have) != 3 or any(w is not None and w != h for w, h in zip(shape, have)):
        want = ", ".join(n if w is None else str(w) for n, w in zip("THD", shape))
        raise ValueError(f"{name} must be ({want}), got {tuple(have)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    st, sh, sd = t.stride()
    if sd != 1 and have[2] > 1:
        raise ValueError(f"the heads of {name} must be contiguous, got strides {t.stride()}")
    # a dimension of one element has no stride to speak of
    return (st if have[0] > 1 else have[1] * have[2]), (sh if have[1] > 1 else have[2])


def _spec(T, D, device, has_k, norm, q_weight, k_weight, cos, sin, positions, layout):
    """Checks the options; (norm, layout, P, rot)."""
    if norm not in KINDS:
        raise ValueError(f"norm must be among {sorted(KINDS)}, not {norm!r}")
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be among {sorted(LAYOUTS)}, not {layout!r}")
    if norm == "none" and not (q_weight is k_weight is None):
        raise ValueError("q_weight and k_weight need a norm")
    if k_weight is not None and not has_k:
        raise ValueError("k_weight without k")
    if q_weight is not None:
        _check_vector(q_weight, "q_weight", D, device)
    if k_weight is not None:
        _check_vector(k_weight, "k_weight", D, device)
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin belong together")
    if cos is None:
        if positions is not None:
            raise ValueError("positions without cos and sin")
        return KINDS[norm], LAYOUTS[layout], 0, 0
    for t, name in ((cos, "cos"), (sin, "sin")):
        if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32:
            raise TypeError(f"{name} must be a float32 tensor")
        if t.dim() != 2 or t.shape != cos.shape or not 1 <= t.shape[1] <= D // 2 \
                or t.device != device or not t.is_contiguous():
            raise ValueError(f"{name} must be (positions, pairs), contiguous, with 1 to {D // 2} "
                             f"pairs on {device}, got {tuple(t.shape)} on {t.device}")
    P = cos.shape[0]
    if positions is None:
        if P < T:
            raise ValueError(f"tables of {P} positions for {T} tokens")
    else:
        if not isinstance(positions, torch.Tensor) or positions.dtype is not torch.int32:
            raise TypeError("positions must be an int32 tensor")
        if positions.shape != (T,) or positions.device != device or not positions.is_contiguous():
            raise ValueError(f"positions must be {T} contiguous entries on {device}")
        if P < 1:
            raise ValueError("tables of no position")
    return KINDS[norm], LAYOUTS[layout], P, 2 * cos.shape[1]


def head_norm(q, k=None, *, norm="rms", q_weight=None, k_weight=None, cos=None, sin=None,
              positions=None, layout="pairs", eps=1e-6, out=None, q_out=None, k_out=None,
              stream=None):
    """(q', k') for q (T, Hq, D) and k (T, Hk, D), float32 or bf16, heads contiguous, any token
    and head strides; k' is None without k.

    norm: 'rms', 'layer' or 'none'.  q_weight, k_weight: D float32.  cos, sin: float32 tables
    (positions, pairs); the pairs may be fewer than D / 2, the rest of a head is not turned.
    layout: which elements make pair i, 'pairs' (2i, 2i + 1) or 'halves' (i, i + pairs).
    positions: T int32 (None: 0, 1, ...); a token whose position the tables do not have counts
    for nothing: its heads are left as they are in q_out and k_out where given, and are zeros
    in tensors made here.  out: 'f32' or 'bf16' (None: q's type).  q_out, k_out: tensors to
    write (q_out may be q, k_out k).  stream: as in ``fp8``."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a 3-D torch tensor, (T, H, D)")
    T, Hq, D = q.shape
    dev = q.device
    ldq, hsq = _check_heads(q, "q", (T, Hq, D), dev)
    Hk, ldk, hsk = 0, 0, 0
    if k is not None:
        ldk, hsk = _check_heads(k, "k", (T, None, D), dev, (q.dtype,))
        Hk = k.shape[1]
    norm, layout, P, rot = _spec(T, D, dev, k is not None, norm, q_weight, k_weight, cos, sin,
                                 positions, layout)
    given = [t for t in (q_out, k_out) if isinstance(t, torch.Tensor)]
    if out is not None and out not in _Y_DTYPES:
        raise ValueError(f"out must be 'f32' or 'bf16', not {out!r}")
    dtype = _Y_DTYPES[out] if out is not None else given[0].dtype if given else q.dtype
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    made, zero = [], 0   # bits of the outputs made here

    def output(t, name, heads, bit):
        nonlocal zero
        if t is None:
            t = _new(stream, dev, (T, heads, D), dtype)
            made.append(t)
            zero |= bit
            return t, heads * D, D
        return (t, *_check_heads(t, name, (T, heads, D), dev, (dtype,)))

    q_out, ldqo, hsqo = output(q_out, "q_out", Hq, 1)
    ldko = hsko = 0
    if k is not None:
        k_out, ldko, hsko = output(k_out, "k_out", Hk, 2)
    at = B._at
    if dtype not in _CODES:
        raise TypeError(f"q_out must be float32 or bfloat16, not {dtype}")
    B.launch(dev, B.lib().asp_head_norm, q.data_ptr(), ldq, hsq, Hq, at(k), ldk, hsk, Hk,
             _CODES[q.dtype], T, D, norm, at(q_weight), at(k_weight), eps, at(cos), at(sin), P, rot,
             layout, at(positions), q_out.data_ptr(), ldqo, hsqo, at(k_out), ldko, hsko,
             _CODES[dtype], zero, B.stream_on(stream, dev))
    _lend(stream, *made)
    return q_out, k_out


def head_norm_backward(dq, dk, q, k=None, *, norm="rms", q_weight=None, k_weight=None, cos=None,
                       sin=None, positions=None, layout="pairs", eps=1e-6, need=None, dq_in=None,
                       dk_in=None, workspace=None, stream=None):
    """Gradients of ``head_norm`` from those of its results: dq and dk (float32 or bf16, one type;
    dk None without k), for its inputs q and k; the options are the forward's.  need: the names
    of the wanted gradients (fields of ``HeadNormGrads``; None: of every given input); the
    others are not computed.  dq_in, dk_in: tensors for the gradients of q and k (of their type;
    heads of tokens that count for nothing are left as they are there and are zeros in tensors
    made here; dq_in may be dq and dk_in dk).  The weights' gradients are float32."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a 3-D torch tensor, (T, H, D)")
    T, Hq, D = q.shape
    dev = q.device
    ldq, hsq = _check_heads(q, "q", (T, Hq, D), dev)
    Hk, ldk, hsk = 0, 0, 0
    if k is not None:
        ldk, hsk = _check_heads(k, "k", (T, None, D), dev, (q.dtype,))
        Hk = k.shape[1]
    norm, layout, P, rot = _spec(T, D, dev, k is not None, norm, q_weight, k_weight, cos, sin,
                                 positions, layout)
    wanted = HeadNormGrads(q, k, q_weight, k_weight)
    if need is not None:
        need = tuple(need)
        for name in need:
            if name not in HeadNormGrads._fields or getattr(wanted, name) is None:
                raise ValueError(f"need names {name!r}: no gradient of a given input")
        wanted = HeadNormGrads(*(t if name in need else None
                                 for name, t in wanted._asdict().items()))
    if dq_in is not None and wanted.dq is None or dk_in is not None and wanted.dk is None:
        raise ValueError("a tensor for a gradient that is not wanted")
    if all(t is None for t in wanted):
        return HeadNormGrads(None, None, None, None)
    lddq = hsdq = lddk = hsdk = 0
    dtype, side_q, side_k = None, wanted.dq is not None or wanted.q_weight is not None, \
        wanted.dk is not None or wanted.k_weight is not None
    if side_q:
        lddq, hsdq = _check_heads(dq, "dq", (T, Hq, D), dev)
        dtype = dq.dtype
    if side_k:
        lddk, hsdk = _check_heads(dk, "dk", (T, Hk, D), dev, _CODES if dtype is None else (dtype,))
        dtype = dk.dtype
    made, zero = [], 0

    def new(shape, kind=torch.float32):
        made.append(_new(stream, dev, shape, kind))
        return made[-1]

    def output(t, name, like, heads, bit):
        nonlocal zero
        if like is None:
            return None, 0, 0
        if t is None:
            zero |= bit
            return new((T, heads, D), q.dtype), heads * D, D
        return (t, *_check_heads(t, name, (T, heads, D), dev, (q.dtype,)))

    dq_in, lddqi, hsdqi = output(dq_in, "dq_in", wanted.dq, Hq, 1)
    dk_in, lddki, hsdki = output(dk_in, "dk_in", wanted.dk, Hk, 2)
    d_qw = None if wanted.q_weight is None else new(D)
    d_kw = None if wanted.k_weight is None else new(D)
    if d_qw is not None or d_kw is not None:
        size = B.asp_head_norm_backward_workspace_bytes(T, Hq, Hk, D)
        if workspace is None:
            workspace = _new(stream, dev, max(size, 256), torch.uint8)
        _check_ws(workspace, size, dev)
    at = B._at
    B.launch(dev, B.lib().asp_head_norm_backward, at(dq) if side_q else None, lddq, hsdq,
             at(dk) if side_k else None, lddk, hsdk, _CODES[dtype], q.data_ptr(), ldq, hsq, Hq, at(k),
             ldk, hsk, Hk, _CODES[q.dtype], T, D, norm, at(q_weight), at(k_weight), eps, at(cos),
             at(sin), P, rot, layout, at(positions), at(dq_in), lddqi, hsdqi, at(dk_in), lddki, hsdki,
             zero, at(d_qw), at(d_kw), at(workspace), 0 if workspace is None else workspace.numel(),
             B.stream_on(stream, dev))
    _lend(stream, *made)
    return HeadNormGrads(dq_in, dk_in, d_qw, d_kw)


def _rows(t):
    """t, or a copy where its heads are not contiguous or strides are not what the library takes."""
    return t if t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


class _HeadNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos, sin, positions, options):
        ctx.set_materialize_grads(False)
        given = dict(q_weight=q_weight, k_weight=k_weight, cos=cos, sin=sin, positions=positions)
        ctx.save_for_backward(q, k, *given.values())
        ctx.options = options
        return head_norm(q, k, **given, **options)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq, dk):
        _no_capture()
        q, k, *tensors = ctx.saved_tensors
        given = dict(zip(("q_weight", "k_weight", "cos", "sin", "positions"), tensors))
        need = [n for n, w in zip(HeadNormGrads._fields, ctx.needs_input_grad) if w]
        grads = dict.fromkeys(HeadNormGrads._fields)
        # a result that is not used gives zeros to what only it reads
        for name, used, t in (("dq", dq, q), ("q_weight", dq, given["q_weight"]), ("dk", dk, k),
                              ("k_weight", dk, given["k_weight"])):
            if name in need and used is None:
                grads[name] = torch.zeros_like(t)
                need.remove(name)
        if need:
            dq, dk = (None if t is None else _rows(t) for t in (dq, dk))
            found = head_norm_backward(dq, dk, q, k, need=need, **given, **ctx.options)
            grads.update({n: getattr(found, n) for n in need})
        return (*(grads[n] for n in HeadNormGrads._fields), None, None, None, None)


class HeadNorm(torch.nn.Module):
    """``head_norm`` with its weights as parameters, differentiable in q, k and the weights.

    q, k: (..., T, H, D), the leading dimensions alike; returns (q', k') of their shapes and
    type (k' None without k; heads of tokens without a position are zeros).  cos, sin:
    (positions, pairs) tables; positions: int32 of the shape of q's dimensions before its
    heads, or of its last one, T (None: 0 .. T - 1).  Gradients are reverse mode;
    forward-mode tangents are refused.  Under a HIP graph capture, gradients are refused:
    capture ``head_norm`` and ``head_norm_backward``, which keep no graph of their own."""

    def __init__(self, head_dim, norm="rms", layout="pairs", eps=1e-6, device=None):
        super().__init__()
        if norm not in KINDS:
            raise ValueError(f"norm must be among {sorted(KINDS)}, not {norm!r}")
        if layout not in LAYOUTS:
            raise ValueError(f"layout must be among {sorted(LAYOUTS)}, not {layout!r}")
        self.head_dim, self.norm, self.layout, self.eps = head_dim, norm, layout, eps

        def parameter():
            return None if norm == "none" else torch.nn.Parameter(torch.ones(head_dim, device=device))

        self.q_weight = parameter()
        self.k_weight = parameter()

    def forward(self, q, k=None, cos=None, sin=None, positions=None):
        for t, name in ((q, "q"), (k, "k")):
            if t is not None and (t.dim() < 3 or t.shape[-1] != self.head_dim):
                raise ValueError(f"{name} must be (..., T, H, {self.head_dim}), got {tuple(t.shape)}")
        if k is not None and k.shape[:-2] != q.shape[:-2]:
            raise ValueError(f"q and k must be of the same tokens, got {tuple(q.shape)}, {tuple(k.shape)}")
        lead = q.shape[:-2]
        if cos is not None and (positions is not None or len(lead) > 1):
            if positions is None:
                positions = torch.arange(lead[-1], dtype=torch.int32, device=q.device)
            elif positions.shape not in (lead, lead[-1:]):
                raise ValueError(f"positions must be {tuple(lead)} or ({lead[-1]},), got "
                                 f"{tuple(positions.shape)}")
            positions = positions.expand(lead).reshape(-1).contiguous()
        flat = [None if t is None else _rows(t.reshape(-1, *t.shape[-2:])) for t in (q, k)]
        weights = [_float32(self.q_weight), None if k is None else _float32(self.k_weight)]
        options = dict(norm=self.norm, layout=self.layout, eps=self.eps)
        leaves = (*flat, *weights, cos, sin)
        _no_forward_mode(*leaves)
        if any(t is not None and t.requires_grad for t in (cos, sin)):
            raise ValueError("the tables cos and sin have no gradient")
        if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in leaves):
            _no_capture()
            q2, k2 = _HeadNorm.apply(*flat, *weights, cos, sin, positions, options)
        else:
            q2, k2 = head_norm(*flat, q_weight=weights[0], k_weight=weights[1], cos=cos, sin=sin,
                               positions=positions, **options)
        return q2.reshape(q.shape), None if k is None else k2.reshape(k.shape)

    def extra_repr(self) -> str:
        return f"{self.head_dim}, norm={self.norm!r}, layout={self.layout!r}, eps={self.eps}"
