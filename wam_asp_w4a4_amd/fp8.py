"""The 8-bit linear layer: E4M3 operands with one power-of-two scale for each
block of 128, for the projections that 4 bits hurt.

``Fp8Layer`` holds a packed weight on the device and, like ``PackedLayer``, a
``forward``; it also has the layer's gradients.  ``quantize`` and ``Fp8Tensor``
are the format itself (``include/asp.h`` describes its bytes): what
``norm.gated_norm`` hands over with ``out="fp8"`` enters ``forward`` as it is.
All arithmetic happens inside libasp.
"""

from __future__ import annotations

import contextlib
from dataclasses import dataclass

import torch

from . import binding as B
from .layer import _Y_DTYPES, _check_ws, _check_y

BLOCK = 128
_NAMES = {torch.float32: "f32", torch.bfloat16: "bf16"}
_CODES = {torch.float32: B.ASP_F32, torch.bfloat16: B.ASP_BF16}
_HERE = contextlib.nullcontext()


def _on(device):
    """The device made current for a launch, where it is not already."""
    if device.type != "cuda" or device.index == torch.cuda.current_device():
        return _HERE
    return torch.cuda.device(device)


def _lend(stream, *tensors):
    """Tensors made here (on torch's current stream) are used on `stream`: the
    allocator is told, so that their memory is not given away too early."""
    if stream is None:
        return
    for t in tensors:
        if t is not None and t.is_cuda:
            t.record_stream(torch.cuda.ExternalStream(stream, t.device))


def _no_capture():
    """Autograd's own bookkeeping of eager leaves does not survive a capture."""
    if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
        raise RuntimeError("gradients under a graph capture: capture the explicit forward and "
                           "backward calls instead of autograd")


def _stride(t):
    """Row stride of a 2-D tensor (of one row: its width; the stride says nothing)."""
    return t.shape[1] if t.shape[0] <= 1 else t.stride(0)


def _check_rows(t, name, rows, cols, device, dtypes=tuple(_NAMES)):
    """t must be a (rows, cols) matrix with contiguous rows that do not overlap."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if t.dim() != 2 or t.shape[1] != cols or (rows is not None and t.shape[0] != rows):
        raise ValueError(f"{name} must be ({'M' if rows is None else rows}, {cols}), "
                         f"got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.numel() and ((cols > 1 and t.stride(1) != 1) or _stride(t) < cols):
        raise ValueError(f"the rows of {name} must be contiguous and apart, "
                         f"got strides {t.stride()}")


def _check_vector(t, name, size, device):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32:
        raise TypeError(f"{name} must be a float32 tensor")
    if tuple(t.shape) != (size,) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be {size} contiguous entries on {device}, "
                         f"got {tuple(t.shape)} on {t.device}")


def _groups(cols):
    return (cols + 4 * BLOCK - 1) // (4 * BLOCK)


def _pitch(cols):
    return (cols + BLOCK - 1) // BLOCK * BLOCK


@dataclass
class Fp8Tensor:
    """A rows x cols matrix in the 8-bit format (blocks along its rows)."""
    rows: int
    cols: int
    codes: torch.Tensor    # rows x P uint8, P = cols rounded up to 128
    scales: torch.Tensor   # ceil(P / 512) x rows x 4 uint8 (E8M0)

    @staticmethod
    def empty(rows, cols, device):
        return Fp8Tensor(rows, cols,
                         torch.empty((rows, _pitch(cols)), dtype=torch.uint8, device=device),
                         torch.empty((_groups(cols), rows, 4), dtype=torch.uint8, device=device))

    def check(self, name="the 8-bit tensor"):
        """Codes and scales are what rows and cols say (the C ABI sees only pointers)."""
        for t, shape in ((self.codes, (self.rows, _pitch(self.cols))),
                         (self.scales, (_groups(self.cols), self.rows, 4))):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8:
                raise TypeError(f"{name}: codes and scales must be uint8 tensors")
            if tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{name}: a {self.rows} x {self.cols} matrix needs contiguous "
                                 f"{shape}, got {tuple(t.shape)}")
        if self.codes.device != self.scales.device:
            raise ValueError(f"{name}: codes on {self.codes.device}, scales on "
                             f"{self.scales.device}")

    def dequantize(self, dtype="f32", stream=None):
        """The values as a float32 or bf16 matrix."""
        self.check()
        if dtype not in _Y_DTYPES:
            raise ValueError(f"dtype must be 'f32' or 'bf16', not {dtype!r}")
        out = torch.empty((self.rows, self.cols), dtype=_Y_DTYPES[dtype],
                          device=self.codes.device)
        with _on(out.device):
            B.asp_fp8_dequantize(self.codes, self.scales, self.rows, self.cols, out,
                                 B.DTYPES[dtype], stream)
        _lend(stream, out)
        return out


def quantize(x, transpose=False, stream=None):
    """x (M x K, float32 or bf16, any row stride) in the 8-bit format; with
    ``transpose`` its transpose (K x M, blocks of 128 of x's rows)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a 2-D torch tensor")
    _check_rows(x, "x", None, x.shape[1], x.device)
    M, K = x.shape
    q = Fp8Tensor.empty(K, M, x.device) if transpose else Fp8Tensor.empty(M, K, x.device)
    call = B.asp_fp8_quantize_t if transpose else B.asp_fp8_quantize
    with _on(x.device):
        call(x, _CODES[x.dtype], M, K, _stride(x), q.codes, q.scales, stream)
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
        _check_rows(w, "w", None, w.shape[1], w.device)
        N, K = w.shape
        if bias is not None:
            _check_vector(bias, "bias", N, w.device)
        q = Fp8Tensor.empty(N, K, w.device)
        t = Fp8Tensor.empty(K, N, w.device) if backward else None
        ct, st = (t.codes, t.scales) if backward else (None, None)
        with _on(w.device):
            B.asp_fp8_quantize_weight(w, _CODES[w.dtype], N, K, _stride(w), q.codes, q.scales,
                                      ct, st, stream)
        _lend(stream, q.codes, q.scales, ct, st)
        return cls(N, K, q.codes, q.scales, ct, st, bias)

    def __post_init__(self):
        Fp8Tensor(self.N, self.K, self.codes, self.scales).check("the weight")
        if (self.codes_t is None) != (self.scales_t is None):
            raise ValueError("codes_t and scales_t belong together")
        if self.codes_t is not None:
            Fp8Tensor(self.K, self.N, self.codes_t, self.scales_t).check("the transposed weight")
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
        ``Fp8Tensor``; y_dtype 'f32' or 'bf16' (None: x's; 'bf16' for codes)."""
        quantised = isinstance(x, Fp8Tensor)
        if quantised:
            x.check("x")
            if x.cols != self.K:
                raise ValueError(f"x must be (M, {self.K}), got ({x.rows}, {x.cols})")
            if x.codes.device != self.device:
                raise ValueError(f"x is on {x.codes.device}, the layer on {self.device}")
            M, y_dtype = x.rows, y_dtype or "bf16"
        else:
            _check_rows(x, "x", None, self.K, self.device)
            M, y_dtype = x.shape[0], y_dtype or _NAMES[x.dtype]
        _check_y(y, M, self.N, y_dtype, self.device)
        size = B.asp_fp8_gemm_workspace_bytes if quantised else B.asp_fp8_workspace_bytes
        need = size(M, self.N, self.K)
        made = []
        if y is None:
            y = torch.empty((M, self.N), dtype=_Y_DTYPES[y_dtype], device=self.device)
            made.append(y)
        if workspace is not None:
            _check_ws(workspace, need, self.device)
        elif need:
            workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
            made.append(workspace)
        have = 0 if workspace is None else workspace.numel()
        with _on(self.device):
            if quantised:
                B.asp_fp8_gemm(x.codes, x.scales, self.codes, self.scales, M, self.N, self.K,
                               self.bias, y, B.DTYPES[y_dtype], workspace, have, stream)
            else:
                B.asp_fp8_forward(x, _CODES[x.dtype], _stride(x), M, self.N, self.K, self.codes,
                                  self.scales, self.bias, y, B.DTYPES[y_dtype], workspace, have,
                                  stream)
        _lend(stream, *made)
        return y

    def backward(self, dy, x=None, need_dx=True, need_db=None, dw_dtype="f32", workspace=None,
                 stream=None):
        """(dx, dw, db) for dy (M x N): dx in dy's type where ``need_dx``, dw (N x K, of
        ``dw_dtype``) where x is given, db float32 where ``need_db`` (None: where the
        layer has a bias); the others are None."""
        _check_rows(dy, "dy", None, self.N, self.device)
        M = dy.shape[0]
        if x is not None:
            _check_rows(x, "x", M, self.K, self.device)
        if dw_dtype not in _Y_DTYPES:
            raise ValueError(f"dw_dtype must be 'f32' or 'bf16', not {dw_dtype!r}")
        if need_dx and self.codes_t is None:
            raise ValueError("dx needs the transposed weight: pack the layer with backward=True")
        dev, made = self.device, []

        def new(shape, dtype):
            made.append(torch.empty(shape, dtype=dtype, device=dev))
            return made[-1]

        dx = new((M, self.K), dy.dtype) if need_dx else None
        dw = new((self.N, self.K), _Y_DTYPES[dw_dtype]) if x is not None else None
        db = new((self.N,), torch.float32) if (self.bias is not None if need_db is None
                                              else need_db) else None
        if dx is None and dw is None and db is None:
            return None, None, None
        need = B.asp_fp8_backward_workspace_bytes(M, self.N, self.K)
        if workspace is not None:
            _check_ws(workspace, need, dev)
        else:
            workspace = new((max(need, 256),), torch.uint8)
        with _on(dev):
            B.asp_fp8_backward(dy, _CODES[dy.dtype], _stride(dy), x,
                               B.ASP_F32 if x is None else _CODES[x.dtype],
                               self.K if x is None else _stride(x), M, self.N, self.K,
                               self.codes_t, self.scales_t, dx, _CODES[dy.dtype], dw,
                               B.DTYPES[dw_dtype], db, workspace, workspace.numel(), stream)
        _lend(stream, *made)
        return dx, dw, db
