"""ctypes binding of libasp's C entry points (argument marshalling only).

Every function has the name and argument order of its C counterpart in
``include/asp.h``.  Array arguments may be torch tensors (device or host,
contiguous) or NumPy arrays (host); ``None`` passes NULL.  The stream argument
defaults to torch's current stream on the tensors' device.  A non-zero status
raises :class:`ASPError` with the library's own message.

The library is loaded on first use; a missing build raises at once -- there is
no fallback implementation.
"""

from __future__ import annotations

import ctypes
import functools
import os
import sys

import numpy as np

ABI_VERSION = 8
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libasp.so")

ASP_F32 = 0
ASP_BF16 = 1
ASP_E4M3 = 2          # asp_norm_gate's n in the 8-bit format
ASP_NORM_NONE, ASP_NORM_RMS, ASP_NORM_LAYER = 0, 1, 2
ASP_ROTATE_PAIRS, ASP_ROTATE_HALVES = 0, 1
DTYPES = {"f32": ASP_F32, "bf16": ASP_BF16}

# name -> (restype, argtypes); mirrors include/asp.h
_i32, _i64, _sz, _p = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p
_psz = ctypes.POINTER(ctypes.c_size_t)
_f32 = ctypes.c_float
SIGNATURES = {
    "asp_abi_version": (_i32, []),
    "asp_source_digest": (ctypes.c_char_p, []),
    "asp_status_string": (ctypes.c_char_p, [_i32]),
    "asp_last_error": (ctypes.c_char_p, []),
    "asp_gemm_kernel_name": (ctypes.c_char_p, [_i64, _i64, _i64]),
    "asp_packed_sizes": (_i32, [_i64, _i64, _i32, _psz, _psz, _psz]),
    "asp_pack_weight": (_i32, [_i64, _i64, _i32, _p, _p, _p, _p, _p, _p, _p, _i32]),
    "asp_pack_weight_shared": (_i32, [_i64, _i64, _i32, _p, _p, _p, _p, _p, _p, _p, _i32]),
    "asp_quantize_nvfp4_host": (_i32, [_p, _i64, _i64, _p, _p]),
    "asp_prep_pack_bytes": (_i32, [_i64, _i32, _psz]),
    "asp_pack_prep": (_i32, [_i64, _i32, _p, _p, _p]),
    "asp_quantize_nvfp4": (_i32, [_p, _i64, _i64, _p, _p, _p]),
    "asp_dequantize_nvfp4": (_i32, [_p, _p, _i64, _i64, _p, _p]),
    "asp_act_prep_workspace_bytes": (_i32, [_i64, _i64, _i32, _psz]),
    "asp_act_prep": (_i32, [_p, _i32, _i64, _i64, _i32, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "asp_act_prep_u": (_i32, [_p, _i32, _i64, _i64, _i32, _p, _p, _sz, _p]),
    "asp_act_prep_q": (_i32, [_p, _i32, _i64, _i64, _i32, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "asp_gemm_lowrank": (_i32, [_p, _p, _p, _i64, _i64, _i64, _i32, _p, _p, _p, _p, _p, _i32, _p]),
    "asp_workspace_bytes": (_i32, [_i64, _i64, _i64, _i32, _psz]),
    "asp_forward": (_i32, [_p, _i32, _i64, _i64, _i64, _i32, _p, _p, _p, _p, _p, _p, _i32,
                           _p, _sz, _p]),
    "asp_smoothing_search_workspace_bytes": (_i32, [_i64, _i64, _i64, _i32, _i32, _psz]),
    "asp_smoothing_search": (_i32, [_p, _i32, _i64, _i64, _p, _p, _i64, _p, _i32, _p, _p, _i32,
                                    _p, _p, _p, _sz, _p]),
    "asp_top_eigenspace_workspace_bytes": (_i32, [_i64, _i32, _i32, _psz]),
    "asp_top_eigenspace_slices": (_i32, [_i64, _i32, ctypes.POINTER(ctypes.c_int32)]),
    "asp_metric_product_partials": (_i32, [_p, _i64, _p, _i32, _p, _p]),
    "asp_top_eigenspace": (_i32, [_p, _i64, _p, _i32, _i32, _i32, _p, _p, _p, _p, _sz, _p]),
    "asp_svdq_packed_sizes": (_i32, [_i64, _i64, _i32, _psz, _psz, _psz, _psz]),
    "asp_svdq_gram": (_i32, [_i64, _i64, _p, _p, _p]),
    "asp_svdq_pack_weight": (_i32, [_i64, _i64, _i32, _p, _p, _p, _p, _p, _p, _p]),
    "asp_svdq_workspace_bytes": (_i32, [_i64, _i64, _i64, _i32, _psz]),
    "asp_svdq_act_quant": (_i32, [_p, _i32, _i64, _i64, _p, _p, _p, _p]),
    "asp_svdq_gemm": (_i32, [_p, _p, _p, _i64, _i64, _i64, _i32, _p, _p, _p, _p, _p, _i32, _p]),
    "asp_svdq_forward": (_i32, [_p, _i32, _i64, _i64, _i32, _p, _p, _p, _p, _p, _i64, _p, _i32,
                                _p, _sz, _p]),
    "asp_forward_noalloc": (_i32, [_p, _i32, _i64, _i64, _i64, _i32, _p, _p, _p, _p, _p, _p,
                                   _i32, _p]),
    "asp_forward_group": (_i32, [_i32, _p, _i32, _i64, _i64, _i32, _p, _p, _p, _p, _p, _p, _p,
                                 _i32, _p, _p, _p]),
    "asp_forward_group_stages": (_i32, [_i32, _i32, _p, _i32, _i64, _i64, _i32, _p, _p, _p, _p,
                                        _p, _p, _p, _i32, _p, _p, _p]),
    "asp_fp8_sizes": (_i32, [_i64, _i64, _psz, _psz]),
    "asp_fp8_quantize": (_i32, [_p, _i32, _i64, _i64, _i64, _p, _p, _p]),
    "asp_fp8_quantize_t": (_i32, [_p, _i32, _i64, _i64, _i64, _p, _p, _p]),
    "asp_fp8_quantize_weight": (_i32, [_p, _i32, _i64, _i64, _i64, _p, _p, _p, _p, _p]),
    "asp_fp8_dequantize": (_i32, [_p, _p, _i64, _i64, _p, _i32, _p]),
    "asp_fp8_gemm_workspace_bytes": (_i32, [_i64, _i64, _i64, _psz]),
    "asp_fp8_gemm": (_i32, [_p, _p, _p, _p, _i64, _i64, _i64, _p, _p, _i32, _p, _sz, _p]),
    "asp_fp8_workspace_bytes": (_i32, [_i64, _i64, _i64, _psz]),
    "asp_fp8_forward": (_i32, [_p, _i32, _i64, _i64, _i64, _i64, _p, _p, _p, _p, _i32, _p, _sz,
                               _p]),
    "asp_fp8_backward_workspace_bytes": (_i32, [_i64, _i64, _i64, _psz]),
    "asp_fp8_backward": (_i32, [_p, _i32, _i64, _p, _i32, _i64, _i64, _i64, _i64, _p, _p, _p, _i32,
                                _p, _i32, _p, _p, _sz, _p]),
    "asp_norm_gate": (_i32, [_p, _i64, _p, _i64, _i32, _i64, _i64, _f32, _i32, _p, _p, _i32, _p,
                             _p, _p, _p, _i64, _i32, _p, _f32, _p, _i64, _p, _i32, _i64, _p,
                             _i32, _p]),
    "asp_norm_gate_backward_workspace_bytes": (_i32, [_i64, _i64, _i32, _psz]),
    "asp_norm_gate_backward": (_i32, [_p, _i64, _p, _i64, _i32, _p, _i64, _p, _i64, _i32, _i64,
                                      _i64, _f32, _i32, _p, _p, _i32, _p, _p, _p, _i64, _i32, _p,
                                      _f32, _p, _i64, _p, _i64, _i32, _p, _p, _p, _p, _p, _p,
                                      _i64, _p, _sz, _p]),
    "asp_head_norm": (_i32, [_p, _i64, _i64, _i32, _p, _i64, _i64, _i32, _i32, _i64, _i32, _i32,
                             _p, _p, _f32, _p, _p, _i64, _i32, _i32, _p, _p, _i64, _i64, _p, _i64,
                             _i64, _i32, _i32, _p]),
    "asp_head_norm_backward_workspace_bytes": (_i32, [_i64, _i32, _i32, _i32, _psz]),
    "asp_head_norm_backward": (_i32, [_p, _i64, _i64, _p, _i64, _i64, _i32, _p, _i64, _i64, _i32,
                                      _p, _i64, _i64, _i32, _i32, _i64, _i32, _i32, _p, _p, _f32,
                                      _p, _p, _i64, _i32, _i32, _p, _p, _i64, _i64, _p, _i64, _i64,
                                      _i32, _p, _p, _p, _sz, _p]),
    "asp_attention_workspace_bytes": (_i32, [_i64, _i64, _i32, _i32, _i32, _i32, _psz]),
    "asp_attention": (_i32, [_p, _i64, _i64, _p, _i64, _i64, _p, _i64, _i64, _i32, _i64, _i64, _i32,
                             _i32, _i32, _f32, _i32, _p, _p, _p, _p, _p, _i64, _i64, _p, _i32, _p,
                             _sz, _p]),
    "asp_attention_backward_workspace_bytes": (_i32, [_i64, _i64, _i32, _i32, _i32, _i32, _psz]),
    "asp_attention_backward": (_i32, [_p, _i64, _i64, _p, _i64, _i64, _p, _i64, _i64, _p, _i64, _i64,
                                      _p, _i64, _i64, _p, _i32, _i64, _i64, _i32, _i32, _i32, _f32,
                                      _i32, _p, _p, _p, _p, _p, _i64, _i64, _p, _i64, _i64, _p, _i64,
                                      _i64, _i32, _p, _sz, _p]),
    "asp_kv_store": (_i32, [_p, _i64, _i64, _p, _i64, _i64, _i32, _i64, _i32, _i32, _i32, _p, _p, _p,
                            _i64, _p, _p, _p, _p, _p]),
    "asp_kv_load": (_i32, [_p, _p, _p, _p, _i64, _i32, _i32, _p, _p, _i32, _p]),
    "asp_attention_cache": (_i32, [_p, _i64, _i64, _i32, _p, _p, _p, _p, _i64, _i64, _i32, _i32, _i32,
                                   _f32, _i32, _p, _p, _p, _p, _p, _i64, _i64, _p, _i32, _p, _sz,
                                   _p]),
}

_lib = None


class ASPError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded libasp.  Raises if it has not been built, if its ABI
    revision differs from this binding's, or if it was built from sources
    other than the ones beside it (a stale build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m wam_asp_w4a4_amd.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        if handle.asp_abi_version() != ABI_VERSION:
            raise RuntimeError("libasp ABI version mismatch")
        from .build import source_digest
        built, current = handle.asp_source_digest().decode(), source_digest()
        if built != current:
            raise RuntimeError(f"{LIB_PATH} was built from other sources (digest {built}, "
                               f"sources {current}): rebuild it with "
                               "`python -m wam_asp_w4a4_amd.build`")
        _lib = handle
    return _lib


def _check(status: int):
    if status != 0:
        msg = lib().asp_last_error().decode()
        raise ASPError(status, msg)


def _ptr(a):
    if a is None:
        return None
    if isinstance(a, np.ndarray):
        if not a.flags["C_CONTIGUOUS"]:
            raise ValueError("NumPy arrays must be C-contiguous")
        return a.ctypes.data
    if not a.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return a.data_ptr()


def _stream(stream, *tensors):
    if stream is not None:
        return stream
    import torch
    for t in tensors:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            return torch.cuda.current_stream(t.device).cuda_stream
    return None


# ------------------------------------------------------------------- host


def asp_abi_version() -> int:
    return lib().asp_abi_version()


def asp_source_digest() -> str:
    return lib().asp_source_digest().decode()


def asp_status_string(status: int) -> str:
    return lib().asp_status_string(status).decode()


def asp_last_error() -> str:
    return lib().asp_last_error().decode()


def asp_packed_sizes(N: int, K: int, r: int):
    c, s, w = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().asp_packed_sizes(N, K, r, ctypes.byref(c), ctypes.byref(s), ctypes.byref(w)))
    return c.value, s.value, w.value


def asp_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().asp_workspace_bytes(M, N, K, r, ctypes.byref(b)))
    return b.value


def asp_prep_pack_bytes(K: int, r: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().asp_prep_pack_bytes(K, r, ctypes.byref(b)))
    return b.value


def asp_pack_prep(K, r, s, v, prep_pack):
    _check(lib().asp_pack_prep(K, r, _ptr(s), _ptr(v), _ptr(prep_pack)))


def asp_pack_weight(N, K, r, w, s, v, w_codes, w_scales, wv, w_prequant=None, n_threads=0):
    _check(lib().asp_pack_weight(N, K, r, _ptr(w), _ptr(s), _ptr(v), _ptr(w_codes),
                                 _ptr(w_scales), _ptr(wv), _ptr(w_prequant), n_threads))


def asp_pack_weight_shared(N, K, r, w, s, v, w_codes, w_scales, wv, w_prequant=None,
                           n_threads=0):
    _check(lib().asp_pack_weight_shared(N, K, r, _ptr(w), _ptr(s), _ptr(v), _ptr(w_codes),
                                        _ptr(w_scales), _ptr(wv), _ptr(w_prequant), n_threads))


def asp_quantize_nvfp4_host(inp, rows, cols, codes, scales):
    _check(lib().asp_quantize_nvfp4_host(_ptr(inp), rows, cols, _ptr(codes), _ptr(scales)))


# ----------------------------------------------------------------- device


def asp_quantize_nvfp4(inp, rows, cols, codes, scales, stream=None):
    _check(lib().asp_quantize_nvfp4(_ptr(inp), rows, cols, _ptr(codes), _ptr(scales),
                                    _stream(stream, inp)))


def asp_dequantize_nvfp4(codes, scales, rows, cols, out, stream=None):
    _check(lib().asp_dequantize_nvfp4(_ptr(codes), _ptr(scales), rows, cols, _ptr(out),
                                      _stream(stream, out)))


def asp_act_prep_workspace_bytes(M: int, K: int, r: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().asp_act_prep_workspace_bytes(M, K, r, ctypes.byref(b)))
    return b.value


def asp_act_prep(x, x_dtype, M, K, r, prep_pack, x_codes, x_scales, u, prequant=None,
                 workspace=None, workspace_bytes=0, stream=None):
    _check(lib().asp_act_prep(_ptr(x), x_dtype, M, K, r, _ptr(prep_pack), _ptr(x_codes),
                              _ptr(x_scales), _ptr(u), _ptr(prequant), _ptr(workspace),
                              workspace_bytes, _stream(stream, x)))


def asp_gemm_kernel_name(M, N, K):
    return lib().asp_gemm_kernel_name(M, N, K).decode()


def asp_act_prep_u(x, x_dtype, M, K, r, prep_pack, workspace=None, workspace_bytes=0,
                   stream=None):
    _check(lib().asp_act_prep_u(_ptr(x), x_dtype, M, K, r, _ptr(prep_pack), _ptr(workspace),
                                workspace_bytes, _stream(stream, x)))


def asp_act_prep_q(x, x_dtype, M, K, r, prep_pack, x_codes, x_scales, u, prequant=None,
                   workspace=None, workspace_bytes=0, stream=None):
    _check(lib().asp_act_prep_q(_ptr(x), x_dtype, M, K, r, _ptr(prep_pack), _ptr(x_codes),
                                _ptr(x_scales), _ptr(u), _ptr(prequant), _ptr(workspace),
                                workspace_bytes, _stream(stream, x)))


def asp_gemm_lowrank(x_codes, x_scales, u, M, N, K, r, w_codes, w_scales, wv, bias, y, y_dtype,
                     stream=None):
    _check(lib().asp_gemm_lowrank(_ptr(x_codes), _ptr(x_scales), _ptr(u), M, N, K, r,
                                  _ptr(w_codes), _ptr(w_scales), _ptr(wv), _ptr(bias), _ptr(y),
                                  y_dtype, _stream(stream, y)))


def asp_smoothing_search_workspace_bytes(M, N, K, r, n_candidates):
    out = ctypes.c_size_t(0)
    _check(lib().asp_smoothing_search_workspace_bytes(M, N, K, r, n_candidates, ctypes.byref(out)))
    return out.value


def asp_smoothing_search(x, x_dtype, M, K, w, bias, N, v, r, alphas, betas, workspace,
                         workspace_bytes, stream=None):
    """Returns (mse per candidate as a NumPy float64 array, best index)."""
    # converted copies are held in locals until the call returns
    alphas = np.ascontiguousarray(alphas, np.float32)
    betas = np.ascontiguousarray(betas, np.float32)
    w = np.ascontiguousarray(w, np.float32)
    bias = None if bias is None else np.ascontiguousarray(bias, np.float32)
    v = None if v is None else np.ascontiguousarray(v, np.float32)
    n = len(alphas)
    mse = np.empty(n, np.float64)
    best = ctypes.c_int32(0)
    _check(lib().asp_smoothing_search(
        _ptr(x), x_dtype, M, K, _ptr(w), _ptr(bias), N, _ptr(v), r, _ptr(alphas), _ptr(betas), n,
        _ptr(mse), ctypes.cast(ctypes.byref(best), ctypes.c_void_p).value, _ptr(workspace),
        workspace_bytes, _stream(stream, x)))
    return mse, int(best.value)


def asp_top_eigenspace_workspace_bytes(K, p, r):
    out = ctypes.c_size_t(0)
    _check(lib().asp_top_eigenspace_workspace_bytes(K, p, r, ctypes.byref(out)))
    return out.value


def asp_top_eigenspace_slices(K, p):
    out = ctypes.c_int32(0)
    _check(lib().asp_top_eigenspace_slices(K, p, ctypes.byref(out)))
    return int(out.value)


def asp_metric_product_partials(g, K, v, p, yp, stream=None):
    _check(lib().asp_metric_product_partials(_ptr(g), K, _ptr(v), p, _ptr(yp),
                                             _stream(stream, g)))


def asp_top_eigenspace(g, K, v0, p, r, iters, v, evals, resid, workspace, workspace_bytes,
                       stream=None):
    _check(lib().asp_top_eigenspace(_ptr(g), K, _ptr(v0), p, r, iters, _ptr(v), _ptr(evals),
                                    _ptr(resid), _ptr(workspace), workspace_bytes,
                                    _stream(stream, g)))


def asp_svdq_packed_sizes(N, K, r):
    """(code bytes, scale bytes, L1 bytes, prep-pack bytes) of one packed layer."""
    out = [ctypes.c_size_t(0) for _ in range(4)]
    _check(lib().asp_svdq_packed_sizes(N, K, r, *[ctypes.byref(o) for o in out]))
    return tuple(o.value for o in out)


def asp_svdq_gram(N, K, w, s, g):
    _check(lib().asp_svdq_gram(N, K, _ptr(w), _ptr(s), _ptr(g)))


def asp_svdq_pack_weight(N, K, r, w, s, v, codes, scales, l1, prep):
    _check(lib().asp_svdq_pack_weight(N, K, r, _ptr(w), _ptr(s), _ptr(v), _ptr(codes),
                                      _ptr(scales), _ptr(l1), _ptr(prep)))


def asp_svdq_workspace_bytes(M, N, K, r):
    out = ctypes.c_size_t(0)
    _check(lib().asp_svdq_workspace_bytes(M, N, K, r, ctypes.byref(out)))
    return out.value


def asp_svdq_act_quant(x, x_dtype, M, K, prep_pack, x_codes, x_scales, stream=None):
    _check(lib().asp_svdq_act_quant(_ptr(x), x_dtype, M, K, _ptr(prep_pack), _ptr(x_codes),
                                    _ptr(x_scales), _stream(stream, x)))


def asp_svdq_gemm(x_codes, x_scales, u, M, N, K, r, w_codes, w_scales, l1, bias, y, y_dtype,
                  stream=None):
    _check(lib().asp_svdq_gemm(_ptr(x_codes), _ptr(x_scales), _ptr(u), M, N, K, r, _ptr(w_codes),
                               _ptr(w_scales), _ptr(l1), _ptr(bias), _ptr(y), y_dtype,
                               _stream(stream, y)))


def asp_svdq_forward(x, x_dtype, M, K, r, prep_pack, w_codes, w_scales, l1, bias, N, y, y_dtype,
                     workspace, workspace_bytes, stream=None):
    _check(lib().asp_svdq_forward(_ptr(x), x_dtype, M, K, r, _ptr(prep_pack), _ptr(w_codes),
                                  _ptr(w_scales), _ptr(l1), _ptr(bias), N, _ptr(y), y_dtype,
                                  _ptr(workspace), workspace_bytes, _stream(stream, x)))


def _ptr_array(items):
    """A host array of device pointers (NULL entries for None); None for a None list."""
    if items is None:
        return None, None
    arr = (ctypes.c_void_p * len(items))(*[_ptr(a) for a in items])
    return arr, ctypes.cast(arr, ctypes.c_void_p).value


def asp_forward_group(x, x_dtype, M, K, r, prep_pack, w_codes, w_scales, wv, bias, N, y, y_dtype,
                      workspace, workspace_bytes, stream=None):
    """Per-layer arguments are equal-length lists (bias and wv may be None)."""
    asp_forward_group_stages(7, x, x_dtype, M, K, r, prep_pack, w_codes, w_scales, wv, bias, N, y,
                             y_dtype, workspace, workspace_bytes, stream)


def asp_forward_group_stages(stages, x, x_dtype, M, K, r, prep_pack, w_codes, w_scales, wv, bias,
                             N, y, y_dtype, workspace, workspace_bytes, stream=None):
    n = len(y)
    keep = []  # the ctypes arrays must outlive the call

    def arr(items):
        a, p = _ptr_array(items)
        keep.append(a)
        return p

    nn = (ctypes.c_int64 * n)(*N)
    nb = (ctypes.c_size_t * n)(*workspace_bytes)
    keep += [nn, nb]
    _check(lib().asp_forward_group_stages(
        stages, n, arr(x), x_dtype, M, K, r, arr(prep_pack), arr(w_codes), arr(w_scales), arr(wv),
        arr(bias), ctypes.cast(nn, ctypes.c_void_p).value, arr(y), y_dtype, arr(workspace),
        ctypes.cast(nb, ctypes.c_void_p).value, _stream(stream, *y)))


def asp_forward_noalloc(x, x_dtype, M, N, K, r, prep_pack, w_codes, w_scales, wv, bias, y,
                        y_dtype, stream=None):
    _check(lib().asp_forward_noalloc(_ptr(x), x_dtype, M, N, K, r, _ptr(prep_pack),
                                     _ptr(w_codes), _ptr(w_scales), _ptr(wv), _ptr(bias), _ptr(y),
                                     y_dtype, _stream(stream, y)))


def asp_forward(x, x_dtype, M, N, K, r, prep_pack, w_codes, w_scales, wv, bias, y, y_dtype,
                workspace, workspace_bytes, stream=None):
    _check(lib().asp_forward(_ptr(x), x_dtype, M, N, K, r, _ptr(prep_pack), _ptr(w_codes),
                             _ptr(w_scales), _ptr(wv), _ptr(bias), _ptr(y), y_dtype,
                             _ptr(workspace), workspace_bytes, _stream(stream, y)))


# ------------------------------------------- 8-bit linear layer, gated norms
#
# Matrices and tables that the C entry points take with a row stride may be
# strided tensors here (their rows contiguous); the stride is an argument.


def _at(a):
    """The address of a tensor of any strides (None: NULL)."""
    return None if a is None else a.data_ptr()


def stream_on(stream, device):
    """The stream handle for a launch on `device`: the caller's, else torch's current one."""
    if stream is not None or device.type != "cuda":
        return stream
    return sys.modules["torch"]._C._cuda_getCurrentRawStream(device.index)


def launch(device, fn, *args):
    """fn(*args) with `device` current, raising the library's error.  For callers that
    have checked their tensors, which lie on `device`, and pass addresses: a kernel given
    the host's would fault."""
    if device.type != "cuda":
        raise ValueError(f"the tensors are on {device}, not on a GPU")
    torch = sys.modules["torch"]   # there, since `device` is one of its
    if device.index == torch._C._cuda_getDevice():
        status = fn(*args)
    else:
        with torch.cuda.device(device):
            status = fn(*args)
    if status:
        _check(status)


@functools.lru_cache(maxsize=4096)
def _size(name, *args):
    """A size that depends on the numbers alone."""
    out = ctypes.c_size_t(0)
    _check(getattr(lib(), name)(*args, ctypes.byref(out)))
    return out.value


def asp_fp8_sizes(rows, cols):
    """(code bytes, scale bytes) of a rows x cols matrix in the 8-bit format."""
    c, s = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().asp_fp8_sizes(rows, cols, ctypes.byref(c), ctypes.byref(s)))
    return c.value, s.value


def asp_fp8_quantize(inp, dtype, rows, cols, ld, codes, scales, stream=None):
    _check(lib().asp_fp8_quantize(_at(inp), dtype, rows, cols, ld, _ptr(codes), _ptr(scales),
                                  _stream(stream, inp)))


def asp_fp8_quantize_t(inp, dtype, rows, cols, ld, codes_t, scales_t, stream=None):
    _check(lib().asp_fp8_quantize_t(_at(inp), dtype, rows, cols, ld, _ptr(codes_t),
                                    _ptr(scales_t), _stream(stream, inp)))


def asp_fp8_quantize_weight(w, dtype, N, K, ld, codes, scales, codes_t=None, scales_t=None,
                            stream=None):
    _check(lib().asp_fp8_quantize_weight(_at(w), dtype, N, K, ld, _ptr(codes), _ptr(scales),
                                         _ptr(codes_t), _ptr(scales_t), _stream(stream, w)))


def asp_fp8_dequantize(codes, scales, rows, cols, out, dtype, stream=None):
    _check(lib().asp_fp8_dequantize(_ptr(codes), _ptr(scales), rows, cols, _ptr(out), dtype,
                                    _stream(stream, out)))


def asp_fp8_gemm_workspace_bytes(M, N, K) -> int:
    return _size("asp_fp8_gemm_workspace_bytes", M, N, K)


def asp_fp8_gemm(a_codes, a_scales, b_codes, b_scales, M, N, K, bias, y, y_dtype, workspace=None,
                 workspace_bytes=0, stream=None):
    _check(lib().asp_fp8_gemm(_ptr(a_codes), _ptr(a_scales), _ptr(b_codes), _ptr(b_scales), M, N,
                              K, _ptr(bias), _ptr(y), y_dtype, _ptr(workspace), workspace_bytes,
                              _stream(stream, y)))


def asp_fp8_workspace_bytes(M, N, K) -> int:
    return _size("asp_fp8_workspace_bytes", M, N, K)


def asp_fp8_forward(x, x_dtype, ldx, M, N, K, w_codes, w_scales, bias, y, y_dtype,
                    workspace=None, workspace_bytes=0, stream=None):
    _check(lib().asp_fp8_forward(_at(x), x_dtype, ldx, M, N, K, _ptr(w_codes), _ptr(w_scales),
                                 _ptr(bias), _ptr(y), y_dtype, _ptr(workspace), workspace_bytes,
                                 _stream(stream, y)))


def asp_fp8_backward_workspace_bytes(M, N, K) -> int:
    return _size("asp_fp8_backward_workspace_bytes", M, N, K)


def asp_fp8_backward(dy, dy_dtype, lddy, x, x_dtype, ldx, M, N, K, wt_codes, wt_scales, dx,
                     dx_dtype, dw, dw_dtype, db, workspace, workspace_bytes, stream=None):
    _check(lib().asp_fp8_backward(_at(dy), dy_dtype, lddy, _at(x), x_dtype, ldx, M, N, K,
                                  _ptr(wt_codes), _ptr(wt_scales), _ptr(dx), dx_dtype, _ptr(dw),
                                  dw_dtype, _ptr(db), _ptr(workspace), workspace_bytes,
                                  _stream(stream, dy)))


def asp_norm_gate(x, ldx, y, ldy, dtype, M, C, alpha, post, post_w, gate, pre, pre_w, pre_b, scale,
                  shift, ldt, G, offsets, eps, h, ldh, n, n_dtype, ldn, n_scales=None, zero=0,
                  stream=None):
    _check(lib().asp_norm_gate(_at(x), ldx, _at(y), ldy, dtype, M, C, alpha, post, _ptr(post_w),
                               _at(gate), pre, _ptr(pre_w), _ptr(pre_b), _at(scale), _at(shift),
                               ldt, G, _ptr(offsets), eps, _at(h), ldh, _at(n), n_dtype, ldn,
                               _ptr(n_scales), zero, _stream(stream, x)))


def asp_norm_gate_backward_workspace_bytes(M, C, G) -> int:
    return _size("asp_norm_gate_backward_workspace_bytes", M, C, G)


def asp_norm_gate_backward(dh, lddh, dn, lddn, dn_dtype, h, ldh, y, ldy, dtype, M, C, alpha, post,
                           post_w, gate, pre, pre_w, pre_b, scale, ldt, G, offsets, eps, dx, lddx,
                           dy, lddy, zero, d_post_w, d_gate, d_pre_w, d_pre_b, d_scale, d_shift, ldd,
                           workspace, workspace_bytes, stream=None):
    _check(lib().asp_norm_gate_backward(
        _at(dh), lddh, _at(dn), lddn, dn_dtype, _at(h), ldh, _at(y), ldy, dtype, M, C, alpha, post,
        _ptr(post_w), _at(gate), pre, _ptr(pre_w), _ptr(pre_b), _at(scale), ldt, G, _ptr(offsets),
        eps, _at(dx), lddx, _at(dy), lddy, zero, _ptr(d_post_w), _at(d_gate), _ptr(d_pre_w),
        _ptr(d_pre_b), _at(d_scale), _at(d_shift), ldd, _ptr(workspace), workspace_bytes,
        _stream(stream, dh, dn)))


# ------------------------------------------------------- a block's attention


def asp_head_norm(q, ldq, hsq, Hq, k, ldk, hsk, Hk, dtype, T, D, norm, q_w, k_w, eps, cosine, sine,
                  P, rot, layout, positions, q_out, ldqo, hsqo, k_out, ldko, hsko, out_dtype, zero=0,
                  stream=None):
    _check(lib().asp_head_norm(_at(q), ldq, hsq, Hq, _at(k), ldk, hsk, Hk, dtype, T, D, norm,
                               _ptr(q_w), _ptr(k_w), eps, _ptr(cosine), _ptr(sine), P, rot, layout,
                               _ptr(positions), _at(q_out), ldqo, hsqo, _at(k_out), ldko, hsko,
                               out_dtype, zero, _stream(stream, q)))


def asp_head_norm_backward_workspace_bytes(T, Hq, Hk, D) -> int:
    return _size("asp_head_norm_backward_workspace_bytes", T, Hq, Hk, D)


def asp_head_norm_backward(dq, lddq, hsdq, dk, lddk, hsdk, d_dtype, q, ldq, hsq, Hq, k, ldk, hsk, Hk,
                           dtype, T, D, norm, q_w, k_w, eps, cosine, sine, P, rot, layout, positions,
                           dq_in, lddqi, hsdqi, dk_in, lddki, hsdki, zero, d_q_w, d_k_w, workspace,
                           workspace_bytes, stream=None):
    _check(lib().asp_head_norm_backward(
        _at(dq), lddq, hsdq, _at(dk), lddk, hsdk, d_dtype, _at(q), ldq, hsq, Hq, _at(k), ldk, hsk, Hk,
        dtype, T, D, norm, _ptr(q_w), _ptr(k_w), eps, _ptr(cosine), _ptr(sine), P, rot, layout,
        _ptr(positions), _at(dq_in), lddqi, hsdqi, _at(dk_in), lddki, hsdki, zero, _ptr(d_q_w),
        _ptr(d_k_w), _ptr(workspace), workspace_bytes, _stream(stream, dq, dk)))


def asp_attention_workspace_bytes(Tq, Tk, Hq, Hk, D, G) -> int:
    return _size("asp_attention_workspace_bytes", Tq, Tk, Hq, Hk, D, G)


def asp_attention(q, ldq, hsq, k, ldk, hsk, v, ldv, hsv, dtype, Tq, Tk, Hq, Hk, D, scale, G, q_offsets,
                  kv_offsets, kv_lengths, key_mask, o, ldo, hso, lse, zero=0, workspace=None,
                  workspace_bytes=0, stream=None):
    _check(lib().asp_attention(
        _at(q), ldq, hsq, _at(k), ldk, hsk, _at(v), ldv, hsv, dtype, Tq, Tk, Hq, Hk, D, scale, G,
        _ptr(q_offsets), _ptr(kv_offsets), _ptr(kv_lengths), _ptr(key_mask), _at(o), ldo, hso,
        _ptr(lse), zero, _ptr(workspace), workspace_bytes, _stream(stream, q)))


def asp_attention_backward_workspace_bytes(Tq, Tk, Hq, Hk, D, G) -> int:
    return _size("asp_attention_backward_workspace_bytes", Tq, Tk, Hq, Hk, D, G)


def asp_attention_backward(dout, lddo, hsdo, q, ldq, hsq, k, ldk, hsk, v, ldv, hsv, o, ldo, hso, lse,
                           dtype, Tq, Tk, Hq, Hk, D, scale, G, q_offsets, kv_offsets, kv_lengths,
                           key_mask, dq, lddq, hsdq, dk, lddk, hsdk, dv, lddv, hsdv, zero, workspace,
                           workspace_bytes, stream=None):
    _check(lib().asp_attention_backward(
        _at(dout), lddo, hsdo, _at(q), ldq, hsq, _at(k), ldk, hsk, _at(v), ldv, hsv, _at(o), ldo, hso,
        _ptr(lse), dtype, Tq, Tk, Hq, Hk, D, scale, G, _ptr(q_offsets), _ptr(kv_offsets),
        _ptr(kv_lengths), _ptr(key_mask), _at(dq), lddq, hsdq, _at(dk), lddk, hsdk, _at(dv), lddv,
        hsdv, zero, _ptr(workspace), workspace_bytes, _stream(stream, dout, k)))


def asp_kv_store(k, ldk, hsk, v, ldv, hsv, dtype, T, Hk, D, G, offsets, kv_offsets, kv_lengths, rows,
                 k_codes, k_scales, v_codes, v_scales, stream=None):
    _check(lib().asp_kv_store(_at(k), ldk, hsk, _at(v), ldv, hsv, dtype, T, Hk, D, G, _ptr(offsets),
                              _ptr(kv_offsets), _ptr(kv_lengths), rows, _ptr(k_codes),
                              _ptr(k_scales), _ptr(v_codes), _ptr(v_scales), _stream(stream, k)))


def asp_kv_load(k_codes, k_scales, v_codes, v_scales, rows, Hk, D, k, v, dtype, stream=None):
    _check(lib().asp_kv_load(_ptr(k_codes), _ptr(k_scales), _ptr(v_codes), _ptr(v_scales), rows, Hk, D,
                             _ptr(k), _ptr(v), dtype, _stream(stream, k, v)))


def asp_attention_cache(q, ldq, hsq, dtype, k_codes, k_scales, v_codes, v_scales, Tq, Tk, Hq, Hk, D,
                        scale, G, q_offsets, kv_offsets, kv_lengths, key_mask, o, ldo, hso, lse, zero=0,
                        workspace=None, workspace_bytes=0, stream=None):
    _check(lib().asp_attention_cache(
        _at(q), ldq, hsq, dtype, _ptr(k_codes), _ptr(k_scales), _ptr(v_codes), _ptr(v_scales), Tq, Tk,
        Hq, Hk, D, scale, G, _ptr(q_offsets), _ptr(kv_offsets), _ptr(kv_lengths), _ptr(key_mask),
        _at(o), ldo, hso, _ptr(lse), zero, _ptr(workspace), workspace_bytes, _stream(stream, q)))
