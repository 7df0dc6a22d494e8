"""The norms around a block: kda_gated_norm, kda_residual_norm and their backward passes, of libkda.so (include/kda.h).

``gated`` follows a mixer (``kda``, ``gdn``, ``linattn``): the rms norm of each head's output with its gate.
``residual`` leads from one block to the next: an optional norm of the block's output, its scale per channel, the
residual's sum, and the norm before the next block.  Argument marshalling only; there is no fallback path.
"""
from __future__ import annotations

import ctypes

import torch

from .kda import KDA_OK, KDAError, _pool, _ptr, _used_here, lib
from .linattn import _bytes, _gpu_index, _On, _raw_stream, _row_strides, _workspace
from .qkrope import _DTYPES

GATES = {"sigmoid": 0, "silu": 1}
NORMS = {None: 0, "none": 0, "rms": 1}


def _code_of(x):
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise ValueError(f"x must be bf16, fp16 or fp32, got {x.dtype}")
    return code


def _check_weights(x, D, **weights):
    for name, w in weights.items():
        if w is not None and (w.dtype is not torch.float32 or w.shape != (D,) or not w.is_contiguous()
                              or w.get_device() != x.get_device()):
            raise ValueError(f"{name} must be a contiguous fp32 [D] tensor on x's device")


def _like(name, t, x, dtype, contiguous=True):
    if t.shape != x.shape or t.dtype is not dtype or t.get_device() != x.get_device() or (
            not t.is_contiguous() if contiguous else t.stride(-1) != 1 and t.shape[-1] != 1):
        raise ValueError(f"{name} must be {'contiguous, ' if contiguous else ''}of x's shape and device and {dtype}, "
                         "with contiguous channels")


def _check_gated(x, gate, weight, activation):
    code = _code_of(x)
    if x.dim() != 4 or (x.stride(3) != 1 and x.shape[3] != 1):
        raise ValueError("x must be [B, T, H, D] with contiguous channels")
    _like("gate", gate, x, x.dtype, contiguous=False)
    _check_weights(x, x.shape[3], weight=weight)
    if activation not in GATES:
        raise ValueError(f"activation must be 'sigmoid' or 'silu', got {activation!r}")
    return (*x.shape, code)


def gated(x, gate, out, *, weight=None, activation="sigmoid", eps=1e-6, stream=None):
    """out = x / sqrt(mean(x^2) + eps) * weight * act(gate) for each token and head (kda_gated_norm).

    x, gate: [B, T, H, D], bf16, fp16 or fp32, views with contiguous channels and strides that are multiples of 16
    bytes; out: contiguous, may be x or gate where that is contiguous; weight: fp32 [D] or None; activation:
    "sigmoid" or "silu".  stream: as in ``linattn.fwd``.
    """
    B, T, H, D, code = _check_gated(x, gate, weight, activation)
    _like("out", out, x, x.dtype)
    index = _gpu_index(x)
    with _On(index):
        st = lib().kda_gated_norm(x.data_ptr(), gate.data_ptr(), _ptr(weight), out.data_ptr(), B, T, H, D, code,
                                  GATES[activation], float(eps), _row_strides(x, gate), _raw_stream(stream, index))
    if st != KDA_OK:
        raise KDAError(st, "kda_gated_norm")


def gated_bwd(x, gate, dout, *, weight=None, activation="sigmoid", eps=1e-6, workspace=None, stream=None):
    """Gradients of ``gated`` from its inputs and dout (contiguous).  Returns a dict: dx, dgate (contiguous, of x's dtype)
    and, with a weight, dweight (fp32 [D]).  stream: as in ``linattn.fwd``."""
    B, T, H, D, code = _check_gated(x, gate, weight, activation)
    _like("dout", dout, x, x.dtype)
    index = _gpu_index(x)
    L = lib()
    with _On(index):
        with _pool(stream):
            r = {"dx": torch.empty(x.shape, dtype=x.dtype, device=index),
                 "dgate": torch.empty(x.shape, dtype=x.dtype, device=index)}
            if weight is not None:
                r["dweight"] = torch.empty(D, dtype=torch.float32, device=index)
        _used_here(stream, index, *r.values())
        need = L.kda_gated_norm_bwd_workspace_size(B, T, H, D, code) if weight is not None else 0
        workspace = _workspace(workspace, need, index, stream)
        st = L.kda_gated_norm_bwd(x.data_ptr(), gate.data_ptr(), _ptr(weight), dout.data_ptr(), r["dx"].data_ptr(),
                                  r["dgate"].data_ptr(), _ptr(r.get("dweight")), B, T, H, D, code, GATES[activation],
                                  float(eps), _row_strides(x, gate), _ptr(workspace), _bytes(workspace),
                                  _raw_stream(stream, index))
    if st != KDA_OK:
        raise KDAError(st, "kda_gated_norm_bwd")
    return r


def _token_strides(x, z):
    if x.is_contiguous() and z.is_contiguous():
        return None
    got = []
    for t in (x, z):
        s, n = t.stride(), t.shape
        got += (s[0] if n[0] > 1 else 0, s[1] if n[1] > 1 else 0)
    return (ctypes.c_int64 * 4)(*got)


def _check_residual(x, z, name, weight, scale, post_norm, post_weight):
    code = _code_of(x)
    if x.dim() != 3 or (x.stride(2) != 1 and x.shape[2] != 1):
        raise ValueError("x must be [B, T, D] with contiguous channels")
    if z.dtype is not x.dtype and z.dtype is not torch.float32:
        raise ValueError(f"{name} must be of x's dtype or fp32")
    _like(name, z, x, z.dtype, contiguous=False)
    _check_weights(x, x.shape[2], weight=weight, scale=scale, post_weight=post_weight)
    if post_norm not in NORMS:
        raise ValueError(f"post_norm must be None or 'rms', got {post_norm!r}")
    return (*x.shape, code, _DTYPES[z.dtype])


def residual(x, residual, out, residual_out, *, weight=None, scale=None, post_norm=None, post_weight=None, eps=1e-6,
             stream=None):
    """The step from one block to the next (kda_residual_norm):

        h = x, or its rms norm times post_weight (post_norm="rms");  y = residual + scale * h;
        residual_out = y in the residual's dtype;  out = y / sqrt(mean(y^2) + eps) * weight, from the unrounded y.

    x: [B, T, D], bf16, fp16 or fp32; residual: of x's dtype or fp32 (views with contiguous channels and strides
    that are multiples of 16 bytes); out: contiguous, of x's dtype, may be x; residual_out: contiguous, of the residual's
    dtype, may be the residual; weight, scale, post_weight: fp32 [D] or None.  stream: as in ``linattn.fwd``.
    """
    B, T, D, code, rcode = _check_residual(x, residual, "residual", weight, scale, post_norm, post_weight)
    _like("out", out, x, x.dtype)
    _like("residual_out", residual_out, x, residual.dtype)
    index = _gpu_index(x)
    with _On(index):
        st = lib().kda_residual_norm(x.data_ptr(), residual.data_ptr(), _ptr(weight), _ptr(scale), _ptr(post_weight),
                                     out.data_ptr(), residual_out.data_ptr(), B, T, D, code, rcode, NORMS[post_norm],
                                     float(eps), _token_strides(x, residual), _raw_stream(stream, index))
    if st != KDA_OK:
        raise KDAError(st, "kda_residual_norm")


def residual_bwd(x, residual_out, dout, dresidual_out=None, *, weight=None, scale=None, post_norm=None, post_weight=None,
                 eps=1e-6, workspace=None, stream=None):
    """Gradients of ``residual`` at the stored residual_out, from dout and dresidual_out (contiguous; None: zero).  Returns a
    dict: dx (of x's dtype), dresidual (of residual_out's) and, for the weights given, dweight, dscale, dpost_weight
    (fp32 [D]).  stream: as in ``linattn.fwd``."""
    B, T, D, code, rcode = _check_residual(x, residual_out, "residual_out", weight, scale, post_norm, post_weight)
    _like("dout", dout, x, x.dtype)
    if dresidual_out is not None:
        _like("dresidual_out", dresidual_out, x, residual_out.dtype)
    index = _gpu_index(x)
    L = lib()
    with _On(index):
        with _pool(stream):
            r = {"dx": torch.empty(x.shape, dtype=x.dtype, device=index),
                 "dresidual": torch.empty(x.shape, dtype=residual_out.dtype, device=index)}
            for name, w in (("dweight", weight), ("dscale", scale), ("dpost_weight", post_weight)):
                if w is not None:
                    r[name] = torch.empty(D, dtype=torch.float32, device=index)
        _used_here(stream, index, *r.values())
        need = L.kda_residual_norm_bwd_workspace_size(B, T, D) if len(r) > 2 else 0
        workspace = _workspace(workspace, need, index, stream)
        st = L.kda_residual_norm_bwd(x.data_ptr(), residual_out.data_ptr(), dout.data_ptr(), _ptr(dresidual_out),
                                     _ptr(weight), _ptr(scale), _ptr(post_weight), r["dx"].data_ptr(),
                                     r["dresidual"].data_ptr(), _ptr(r.get("dweight")), _ptr(r.get("dscale")),
                                     _ptr(r.get("dpost_weight")), B, T, D, code, rcode, NORMS[post_norm], float(eps),
                                     _token_strides(x, residual_out), _ptr(workspace), _bytes(workspace),
                                     _raw_stream(stream, index))
    if st != KDA_OK:
        raise KDAError(st, "kda_residual_norm_bwd")
    return r
