"""The 8-bit linear layer: E4M3 operands with one power-of-two scale for each
block of 128, for the projections that 4 bits hurt.

``Fp8Layer`` holds a packed weight on the device and, like ``PackedLayer``, a
``forward``; it also has the layer's gradients.  ``quantize`` and ``Fp8Tensor``
are the format itself (``include/asp.h`` describes its bytes): what
``norm.gated_norm`` hands over with ``out="fp8"`` enters ``forward`` as it is.
All arithmetic happens inside libasp.

Calls run on torch's current stream, or on ``stream`` (a handle): inputs, and outputs
and workspaces that are given, must be ready for it.  What such a call makes belongs to
``stream``: the current one waits for it before it reads them.
"""

from __future__ import annotations

from dataclasses import dataclass

import torch
from torch.autograd import forward_ad

from . import binding as B
from .layer import _Y_DTYPES, _check_ws, _check_y, _lend, _made_for, _new

BLOCK = 128
_NAMES = {torch.float32: "f32", torch.bfloat16: "bf16"}
_CODES = {torch.float32: B.ASP_F32, torch.bfloat16: B.ASP_BF16}


def _no_capture():
    """Refused, since one case ends the process: a backward pass captured while an eager
    graph of the same leaves still lives (their gradients are accumulated on the stream
    that the eager graph noted, which is not being captured)."""
    if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
        raise RuntimeError("gradients under a graph capture: capture the explicit forward and "
                           "backward calls instead of autograd")


def _no_forward_mode(*tensors):
    """The modules' derivatives are reverse mode: a tangent would be lost without a word."""
    if forward_ad._current_level >= 0 and any(
            t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise RuntimeError("no forward-mode derivative: the layer's gradients are reverse mode only")


def _stride(t):
    """Row stride of a 2-D tensor (of one row: its width; the stride says nothing)."""
    return t.shape[1] if t.shape[0] <= 1 else t.stride(0)


def _row_major(t):
    """t itself, or a copy where its rows overlap (a broadcast) or are not contiguous."""
    if t.shape[-1] > 1 and t.stride(-1) != 1 or t.dim() == 2 and _stride(t) < t.shape[1]:
        return t.contiguous()
    return t


def _float32(t):
    return t if t is None or t.dtype is torch.float32 else t.float()


def _check_rows(t, name, rows, cols, device, dtypes=_CODES):
    """t must be a (rows, cols) matrix with contiguous rows that do not overlap (rows
    None: any number).  Returns its row stride."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.device == device:
        shape = t.shape
        if len(shape) == 2 and shape[1] == cols and (rows is None or shape[0] == rows):
            if t.is_contiguous():
                return cols
            ld = _stride(t)
            if (cols == 1 or t.stride(1) == 1) and ld >= cols:
                return ld
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if t.dim() != 2 or t.shape[1] != cols or (rows is not None and t.shape[0] != rows):
        raise ValueError(f"{name} must be ({'M' if rows is None else rows}, {cols}), "
                         f"got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    raise ValueError(f"the rows of {name} must be contiguous and apart, got strides {t.stride()}")


def _check_vector(t, name, size, device):
    if isinstance(t, torch.Tensor) and t.dtype is torch.float32 and t.shape == (size,) \
            and t.device == device and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32:
        raise TypeError(f"{name} must be a float32 tensor")
    raise ValueError(f"{name} must be {size} contiguous entries on {device}, "
                     f"got {tuple(t.shape)} on {t.device}")


def _check_format(rows, cols, codes, scales, name):
    """Codes and scales of a rows x cols matrix (the C ABI sees only pointers)."""
    blocks = (cols + BLOCK - 1) // BLOCK
    want = ((rows, blocks * BLOCK), ((blocks + 3) // 4, rows, 4))
    if isinstance(codes, torch.Tensor) and isinstance(scales, torch.Tensor) \
            and codes.dtype is torch.uint8 and scales.dtype is torch.uint8 \
            and codes.shape == want[0] and scales.shape == want[1] \
            and codes.is_contiguous() and scales.is_contiguous() \
            and codes.device == scales.device:
        return
    for t, shape in zip((codes, scales), want):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8:
            raise TypeError(f"{name}: codes and scales must be uint8 tensors")
        if t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name}: a {rows} x {cols} matrix needs contiguous {shape}, "
                             f"got {tuple(t.shape)}")
    raise ValueError(f"{name}: codes on {codes.device}, scales on {scales.device}")


@dataclass
class Fp8Tensor:
    """A rows x cols matrix in the 8-bit format (blocks along its rows)."""
    rows: int
    cols: int
    codes: torch.Tensor    # rows x P uint8, P = cols rounded up to 128
    scales: torch.Tensor   # ceil(P / 512) x rows x 4 uint8 (E8M0)

    @staticmethod
    def empty(rows, cols, device):
        blocks = (cols + BLOCK - 1) // BLOCK
        return Fp8Tensor(rows, cols,
                         torch.empty((rows, blocks * BLOCK), dtype=torch.uint8, device=device),
                         torch.empty(((blocks + 3) // 4, rows, 4), dtype=torch.uint8,
                                     device=device))

    def check(self, name="the 8-bit tensor"):
        """Codes and scales are what rows and cols say."""
        _check_format(self.rows, self.cols, self.codes, self.scales, name)

    def dequantize(self, dtype="f32", stream=None):
        """The values as a float32 or bf16 matrix."""
        self.check()
        if dtype not in _Y_DTYPES:
            raise ValueError(f"dtype must be 'f32' or 'bf16', not {dtype!r}")
        dev = self.codes.device
        out = _new(stream, dev, (self.rows, self.cols), _Y_DTYPES[dtype])
        B.launch(dev, B.lib().asp_fp8_dequantize, self.codes.data_ptr(), self.scales.data_ptr(),
                 self.rows, self.cols, out.data_ptr(), B.DTYPES[dtype], B.stream_on(stream, dev))
        _lend(stream, out)
        return out


def quantize(x, transpose=False, stream=None):
    """x (M x K, float32 or bf16, any row stride) in the 8-bit format; with
    ``transpose`` its transpose (K x M, blocks of 128 of x's rows)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a 2-D torch tensor")
    M, K = x.shape
    dev = x.device
    ld = _check_rows(x, "x", M, K, dev)
    with _made_for(stream, dev):
        q = Fp8Tensor.empty(K, M, dev) if transpose else Fp8Tensor.empty(M, K, dev)
    fn = B.lib().asp_fp8_quantize_t if transpose else B.lib().asp_fp8_quantize
    B.launch(dev, fn, x.data_ptr(), _CODES[x.dtype], M, K, ld, q.codes.data_ptr(),
             q.scales.data_ptr(), B.stream_on(stream, dev))
    _lend(stream, q.codes, q.scales)
    return q


@dataclass
class Fp8Layer:
    """One linear layer with its weight in the 8-bit format, blocks of 128 x 128."""
    N: int
    K: int
    codes: torch.Tensor             # N x P(K) uint8
    scales: torch.Tensor            # ceil(P(K) / 512) x N x 4 uint8
    codes_t: torch.Tensor | None    # the transposed weight (K x N), for dx
    scales_t: torch.Tensor | None
    bias: torch.Tensor | None       # N float32

    @classmethod
    def pack(cls, w, bias=None, backward=True, stream=None):
        """Pack the device weight w (N x K, float32 or bf16); ``backward`` keeps the
        transposed codes too, which dx needs."""
        if not isinstance(w, torch.Tensor) or w.dim() != 2:
            raise ValueError("w must be a 2-D torch tensor")
        N, K = w.shape
        dev = w.device
        ld = _check_rows(w, "w", N, K, dev)
        if bias is not None:
            _check_vector(bias, "bias", N, w.device)
        with _made_for(stream, dev):
            q = Fp8Tensor.empty(N, K, dev)
            t = Fp8Tensor.empty(K, N, dev) if backward else None
        ct, st = (t.codes, t.scales) if backward else (None, None)
        B.launch(dev, B.lib().asp_fp8_quantize_weight, w.data_ptr(), _CODES[w.dtype], N, K, ld,
                 q.codes.data_ptr(), q.scales.data_ptr(), B._at(ct), B._at(st),
                 B.stream_on(stream, dev))
        _lend(stream, q.codes, q.scales, ct, st)
        return cls(N, K, q.codes, q.scales, ct, st, bias)

    def __post_init__(self):
        _check_format(self.N, self.K, self.codes, self.scales, "the weight")
        if (self.codes_t is None) != (self.scales_t is None):
            raise ValueError("codes_t and scales_t belong together")
        if self.codes_t is not None:
            _check_format(self.K, self.N, self.codes_t, self.scales_t, "the transposed weight")
            if self.codes_t.device != self.codes.device:
                raise ValueError("the transposed weight is on another device")
        if self.bias is not None:
            _check_vector(self.bias, "bias", self.N, self.codes.device)

    @property
    def device(self) -> torch.device:
        return self.codes.device

    def workspace(self, M: int, backward=False) -> torch.Tensor:
        """A workspace that ``forward`` (or ``backward``) of M rows accepts."""
        size = B.asp_fp8_backward_workspace_bytes if backward else B.asp_fp8_workspace_bytes
        return torch.empty(max(size(M, self.N, self.K), 256), dtype=torch.uint8,
                           device=self.device)

    def forward(self, x, y_dtype=None, workspace=None, y=None, stream=None):
        """y = Q(x) W^T + bias for x (M x K, float32 or bf16, any row stride) or an
        ``Fp8Tensor``; y_dtype 'f32' or 'bf16' (None: x's; 'bf16' for codes).  A float32 y
        has float32 sums; a bf16 one is computed at twice the rate, with each 8 consecutive
        products added in 14 bits below their largest (1.5e-5 of y's 2-norm)."""
        dev, N, K = self.codes.device, self.N, self.K
        quantised = isinstance(x, Fp8Tensor)
        if quantised:
            x.check("x")
            if x.cols != K:
                raise ValueError(f"x must be (M, {K}), got ({x.rows}, {x.cols})")
            if x.codes.device != dev:
                raise ValueError(f"x is on {x.codes.device}, the layer on {dev}")
            M, y_dtype = x.rows, y_dtype or "bf16"
            need = B.asp_fp8_gemm_workspace_bytes(M, N, K)
        else:
            ld = _check_rows(x, "x", None, K, dev)
            M, y_dtype = x.shape[0], y_dtype or _NAMES[x.dtype]
            need = B.asp_fp8_workspace_bytes(M, N, K)
        made = None
        if y is not None or y_dtype not in _Y_DTYPES:
            _check_y(y, M, N, y_dtype, dev)
        else:
            made = y = _new(stream, dev, (M, N), _Y_DTYPES[y_dtype])
        have, ws = need, None
        if workspace is not None:
            _check_ws(workspace, need, dev)
            have, ws = workspace.numel(), workspace.data_ptr()
        elif need:
            workspace = _new(stream, dev, need, torch.uint8)
            ws = workspace.data_ptr()
        bias = self.bias
        if bias is not None:
            # a parameter may have been converted since it was checked
            if bias.dtype is not torch.float32 or bias.device != dev or bias.numel() != N:
                _check_vector(bias, "bias", N, dev)
            bias = bias.data_ptr()
        wc, wsc, to = self.codes.data_ptr(), self.scales.data_ptr(), B.stream_on(stream, dev)
        if quantised:
            B.launch(dev, B.lib().asp_fp8_gemm, x.codes.data_ptr(), x.scales.data_ptr(), wc, wsc, M,
                     N, K, bias, y.data_ptr(), B.DTYPES[y_dtype], ws, have, to)
        else:
            B.launch(dev, B.lib().asp_fp8_forward, x.data_ptr(), _CODES[x.dtype], ld, M, N, K, wc,
                     wsc, bias, y.data_ptr(), B.DTYPES[y_dtype], ws, have, to)
        if stream is not None:
            _lend(stream, made)
        return y

    def backward(self, dy, x=None, need_dx=True, need_db=None, dw_dtype="f32", workspace=None,
                 stream=None, dx_dtype=None):
        """(dx, dw, db) for dy (M x N): dx of ``dx_dtype`` (None: dy's type) where
        ``need_dx``, dw (N x K, of ``dw_dtype``) where x is given, db float32 where
        ``need_db`` (None: where the layer has a bias); the others are None.  The types
        choose the arithmetic, as in ``forward``."""
        dev, N, K = self.codes.device, self.N, self.K
        lddy, ldx = _check_rows(dy, "dy", None, N, dev), K
        M = dy.shape[0]
        if x is not None:
            ldx = _check_rows(x, "x", M, K, dev)
        dx_dtype = dx_dtype or _NAMES[dy.dtype]
        if dw_dtype not in _Y_DTYPES or dx_dtype not in _Y_DTYPES:
            raise ValueError(f"dx_dtype and dw_dtype must be 'f32' or 'bf16', not {dx_dtype!r}, "
                             f"{dw_dtype!r}")
        if need_dx and self.codes_t is None:
            raise ValueError("dx needs the transposed weight: pack the layer with backward=True")
        if need_db is None:
            need_db = self.bias is not None
        if not need_dx and x is None and not need_db:
            return None, None, None
        need = B.asp_fp8_backward_workspace_bytes(M, N, K)
        if workspace is not None:
            _check_ws(workspace, need, dev)
        else:
            workspace = _new(stream, dev, need, torch.uint8)
        dx = _new(stream, dev, (M, K), _Y_DTYPES[dx_dtype]) if need_dx else None
        dw = None if x is None else _new(stream, dev, (N, K), _Y_DTYPES[dw_dtype])
        db = _new(stream, dev, N) if need_db else None
        at = B._at
        B.launch(dev, B.lib().asp_fp8_backward, dy.data_ptr(), _CODES[dy.dtype], lddy, at(x),
                 B.ASP_F32 if x is None else _CODES[x.dtype], ldx, M, N, K, at(self.codes_t),
                 at(self.scales_t), at(dx), B.DTYPES[dx_dtype], at(dw), B.DTYPES[dw_dtype], at(db),
                 workspace.data_ptr(), workspace.numel(), B.stream_on(stream, dev))
        _lend(stream, dx, dw, db)
        return dx, dw, db
