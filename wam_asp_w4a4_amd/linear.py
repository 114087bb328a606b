"""A quantised linear module and an all-or-nothing installer.

The model card ("FastWAM UR3 3-task -- 4-bit quantisations", section
"Running the NVFP4 checkpoint") installs its NVFP4 deflated-ASP linears into a
model with one call that refuses to swap only part of the targets.  Here:

* ``ASPLinear`` holds one packed layer (``PackedLayer``) and applies it to an
  input of any leading shape (..., K); y has x's dtype (bfloat16 or float32).
* ``install(model, layers)`` replaces named ``torch.nn.Linear`` submodules by
  ``ASPLinear`` modules.  Every target is validated first -- the name resolves
  to an ``nn.Linear``, the packed layer's K and N equal its in/out features,
  its bias is present exactly when the Linear has one, it sits on the model's
  device -- and only when all of them pass is any module swapped.  Otherwise
  ``InstallError`` lists every problem and the model is left unchanged.
* ``Fp8Linear`` is the same around a layer in the 8-bit format (``fp8.Fp8Layer``),
  for the projections that 4 bits hurt; ``install`` takes either kind.

All arithmetic runs in libasp; this module only reshapes and dispatches.
"""

from __future__ import annotations

from dataclasses import replace
from typing import Mapping

import torch

from .fp8 import _NAMES, Fp8Layer, _float32, _no_capture, _no_forward_mode, _row_major
from .layer import PackedLayer


class InstallError(ValueError):
    """Raised by install() before any module is swapped; .problems lists why."""

    def __init__(self, problems):
        super().__init__("install: no layer swapped:\n  " + "\n  ".join(problems))
        self.problems = list(problems)


class ASPLinear(torch.nn.Module):
    """y = the deflated-ASP NVFP4 layer applied to x (..., in_features).

    The packed weight, scales, low-rank factor, prep constants and bias are
    held as buffers of the packed layer (device tensors); the module has no
    trainable parameters.  Inputs in bfloat16 give bfloat16 outputs, float32
    inputs float32 outputs."""

    def __init__(self, packed: PackedLayer):
        super().__init__()
        self.packed = packed
        self.in_features = packed.K
        self.out_features = packed.N
        self.rank = packed.r

    @classmethod
    def from_linear(cls, linear: torch.nn.Linear, s, v, device=None, form: str = "deflated"):
        """Pack an nn.Linear's weight (and bias) with smoothing vector s (K) and
        basis v (K x r, or None for rank 0)."""
        w = linear.weight.detach().float().cpu().numpy()
        b = None if linear.bias is None else linear.bias.detach().float().cpu().numpy()
        dev = linear.weight.device if device is None else device
        return cls(PackedLayer.pack(w, s, v, b, dev, form=form))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.in_features:
            raise ValueError(f"x has {x.shape[-1]} features, the layer {self.in_features}")
        lead = x.shape[:-1]
        x2 = x.reshape(-1, self.in_features).contiguous()
        y_dtype = "bf16" if x.dtype == torch.bfloat16 else "f32"
        y = self.packed.forward(x2, y_dtype)
        return y.reshape(*lead, self.out_features)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, "
                f"rank={self.rank}, bias={self.packed.bias is not None}, NVFP4 W4A4")


class _Fp8Apply(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, layer, y_dtype):
        ctx.layer = layer
        # the inputs' types; autograd rounds gradients that have more bits
        ctx.dx_dtype = "f32" if y_dtype == "f32" else _NAMES[x.dtype]
        ctx.dw_dtype = "f32" if weight is None or y_dtype == "f32" else _NAMES[weight.dtype]
        ctx.save_for_backward(x if weight is not None and ctx.needs_input_grad[1] else None)
        return layer.forward(x, y_dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        _no_capture()
        x, = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = ctx.layer.backward(dy.contiguous(), x, need_dx=need[0], need_db=need[2],
                                        dw_dtype=ctx.dw_dtype, dx_dtype=ctx.dx_dtype)
        return dx, dw, db, None, None


class Fp8Linear(torch.nn.Module):
    """y = the 8-bit linear layer applied to x (..., in_features), in x's type or the given
    ``y_dtype``: 'f32' has float32 sums in y and all gradients, also for a bf16 x or weight,
    at half the rate (``Fp8Layer.forward`` has the arithmetic).

    Around a packed ``Fp8Layer`` the weight is frozen, and x (and a bias that requires
    it) has a gradient.  With ``weight`` (N x K, float32 or bf16, a parameter) every
    forward packs the weight as it stands, and it has a gradient too: training in
    8-bit products with the optimiser's weight kept in its own type.  Gradients are
    reverse mode; forward-mode tangents are refused.  Under a HIP graph capture, gradients
    are refused: capture ``Fp8Layer.forward`` and ``backward``, which keep no graph of
    their own."""

    def __init__(self, packed: Fp8Layer | None = None, weight=None, bias=None, y_dtype=None):
        super().__init__()
        if (packed is None) == (weight is None):
            raise ValueError("either a packed layer or a weight")
        if packed is not None and bias is not None:
            raise ValueError("a packed layer has its own bias")
        if y_dtype not in (None, "f32", "bf16"):
            raise ValueError(f"y_dtype must be 'f32', 'bf16' or None, not {y_dtype!r}")
        self.packed = packed
        self.y_dtype = y_dtype
        self.weight = weight
        self.bias = packed.bias if packed is not None else bias
        self.out_features, self.in_features = ((packed.N, packed.K) if packed is not None
                                               else weight.shape)

    @classmethod
    def from_linear(cls, linear: torch.nn.Linear, trainable: bool = False, y_dtype=None):
        """From an nn.Linear on the device: its weight packed once, or with ``trainable``
        shared as the parameter that every forward packs.  The bias is kept in float32."""
        bias = None if linear.bias is None else linear.bias.detach().float().contiguous()
        if trainable:
            return cls(weight=linear.weight, y_dtype=y_dtype,
                       bias=None if bias is None else torch.nn.Parameter(bias.clone()))
        return cls(Fp8Layer.pack(linear.weight.detach(), bias), y_dtype=y_dtype)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.in_features:
            raise ValueError(f"x has {x.shape[-1]} features, the layer {self.in_features}")
        x2 = _row_major(x.reshape(-1, self.in_features))
        leaves = (x2, self.weight, self.bias)
        _no_forward_mode(*leaves)
        grads = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in leaves)
        if grads:
            _no_capture()
        layer = self.packed
        if layer is None:
            bias = None if self.bias is None else _float32(self.bias.detach())
            layer = Fp8Layer.pack(self.weight.detach(), bias, backward=grads and x2.requires_grad)
        elif self.bias is not layer.bias or self.bias is not None and self.bias.dtype != torch.float32:
            layer = replace(layer, bias=None if self.bias is None else _float32(self.bias.detach()))
        if grads:
            y = _Fp8Apply.apply(x2, self.weight, self.bias, layer, self.y_dtype)
        else:
            y = layer.forward(x2, self.y_dtype)
        return y.reshape(*x.shape[:-1], self.out_features)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, "
                f"bias={self.bias is not None}, E4M3 block 128, "
                f"{'frozen' if self.weight is None else 'trainable'}")


def _resolve(model: torch.nn.Module, name: str):
    """(parent module, attribute name, module) of a dotted submodule name."""
    parts = name.split(".")
    parent = model
    for p in parts[:-1]:
        parent = getattr(parent, p, None)
        if parent is None:
            return None, parts[-1], None
    return parent, parts[-1], getattr(parent, parts[-1], None)


def install(model: torch.nn.Module, layers: Mapping[str, PackedLayer | Fp8Layer]) -> list:
    """Swap every named nn.Linear of ``model`` for an ASPLinear (or Fp8Linear) of
    its packed layer, or none of them.  Returns the names swapped."""
    problems = []
    plan = []
    for name, packed in layers.items():
        parent, attr, mod = _resolve(model, name)
        if mod is None:
            problems.append(f"{name}: no such submodule")
            continue
        if not isinstance(mod, torch.nn.Linear):
            problems.append(f"{name}: a {type(mod).__name__}, not an nn.Linear")
            continue
        if not isinstance(packed, (PackedLayer, Fp8Layer)):
            problems.append(f"{name}: the packed layer is a {type(packed).__name__}")
            continue
        if (packed.K, packed.N) != (mod.in_features, mod.out_features):
            problems.append(f"{name}: packed {packed.K} -> {packed.N}, Linear "
                            f"{mod.in_features} -> {mod.out_features}")
        if (packed.bias is None) != (mod.bias is None):
            problems.append(f"{name}: bias {'missing' if packed.bias is None else 'unexpected'} "
                            "in the packed layer")
        if packed.device != mod.weight.device:
            problems.append(f"{name}: packed on {packed.device}, the Linear on {mod.weight.device}")
        plan.append((parent, attr, packed))
    if problems:
        raise InstallError(problems)
    for parent, attr, packed in plan:
        setattr(parent, attr, Fp8Linear(packed) if isinstance(packed, Fp8Layer)
                else ASPLinear(packed))
    return list(layers)
