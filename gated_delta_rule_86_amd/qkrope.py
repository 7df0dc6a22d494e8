"""Normalisation of queries and keys for each head with the position rotation in the same pass, and its
backward pass: kda_qk_rope and kda_qk_rope_bwd of libkda.so (include/kda.h).

It prepares q and k for ``linattn``, and for ``kda`` with use_qk_l2norm_in_kernel=False.
``inv_freq`` makes the table of frequencies, also scaled for contexts longer than those trained on.
Argument marshalling only; there is no fallback path.
"""
from __future__ import annotations

import math

import torch

from .kda import KDA_OK, KDAError, _pool, _ptr, _used_here, lib
from .linattn import _bytes, _gpu_index, _On, _raw_stream, _row_strides, _workspace

NORMS = {None: 0, "none": 0, "rms": 1, "l2": 2}
_DTYPES = {torch.bfloat16: 1, torch.float32: 2, torch.float16: 3}


def inv_freq(rotary_dim, base=10000.0, *, scaling=None, factor=1.0, original_context=None, beta_fast=32.0,
             beta_slow=1.0, device=None):
    """Angular frequencies (fp32 [rotary_dim / 2], radians per position) and the attention factor.

    f_i = base^(-2 i / rotary_dim), computed in fp64.  scaling stretches the positions that a model can tell
    apart by ``factor``:
      None      as above;
      "linear"  f / factor: every position moves closer together;
      "ntk"     base * factor^(R / (R - 2)): the highest frequency stays, the lowest is divided by factor;
      "yarn"    a pair that turns more than beta_fast times over original_context positions stays, one
                that turns less than beta_slow times is divided by factor, a linear ramp over
                the pair's index between; the attention factor is 0.1 ln(factor) + 1.
    """
    R = int(rotary_dim)
    if R < 0 or R % 2:
        raise ValueError("rotary_dim must be even and not negative")
    if not base > 1.0:
        raise ValueError("base must be above 1")
    if not factor >= 1.0:
        raise ValueError("factor must be at least 1")
    i = torch.arange(0, R, 2, dtype=torch.float64)
    attention_factor = 1.0
    if scaling == "ntk":
        if R <= 2:
            raise ValueError("ntk scaling needs rotary_dim > 2")
        base = base * factor ** (R / (R - 2))
    f = float(base) ** (-i / max(R, 1))
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if not original_context or original_context < 1:
            raise ValueError("yarn scaling needs original_context")

        def pair_of(turns):  # the (real) index of the pair that turns so often over the context
            return R * math.log(original_context / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo = max(math.floor(pair_of(beta_fast)), 0)
        hi = min(math.ceil(pair_of(beta_slow)), R - 1)  # behind the last pair where all of them turn more often
        ramp = ((torch.arange(R // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - ramp) + f / factor * ramp
        attention_factor = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device=device, dtype=torch.float32), attention_factor


def _check(q, k, positions, inv_freq, norm, q_weight, k_weight, like_q, like_k):
    qs, ks = q.shape, k.shape
    if len(qs) != 4 or len(ks) != 4 or ks[0] != qs[0] or ks[1] != qs[1] or ks[3] != qs[3]:
        raise ValueError("q must be [B, T, Hq, D] and k [B, T, Hk, D]")
    dtype, at = q.dtype, q.get_device()
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"q and k must be bf16, fp16 or fp32, got {dtype}")
    B, T, Hq, D = qs
    for t, shape in ((q, qs), (k, ks), (like_q, qs), (like_k, ks)):
        if t.shape != shape or t.dtype is not dtype or t.get_device() != at or (t.stride(3) != 1 and D != 1):
            raise ValueError("k, and the outputs or gradients of q's and k's shapes, must be of q's dtype and device, "
                             "all with contiguous channels")
    if positions is not None and (positions.dtype is not torch.int64 or positions.shape != (B, T)
                                  or not positions.is_contiguous() or positions.get_device() != at):
        raise ValueError("positions must be a contiguous int64 [B, T] tensor on q's device")
    R = 0
    if inv_freq is not None:
        if (inv_freq.dtype is not torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous()
                or inv_freq.get_device() != at):
            raise ValueError("inv_freq must be a contiguous fp32 [rotary_dim / 2] tensor on q's device")
        R = 2 * inv_freq.numel()
    if norm not in NORMS:
        raise ValueError(f"norm must be one of None, 'rms', 'l2', got {norm!r}")
    for w in (q_weight, k_weight):
        if w is not None and (w.dtype is not torch.float32 or w.shape != (D,) or not w.is_contiguous()
                              or w.get_device() != at):
            raise ValueError("q_weight and k_weight must be contiguous fp32 [D] tensors on q's device")
    return B, T, Hq, ks[2], D, R, code


def fwd(q, k, positions, inv_freq, q_out, k_out, *, q_weight=None, k_weight=None, norm="rms", eps=1e-6,
        interleaved=False, attention_factor=1.0, stream=None):
    """Normalised and rotated q and k, written into ``q_out`` and ``k_out`` (kda_qk_rope).

    q, q_out: [B, T, Hq, D]; k, k_out: [B, T, Hk, D]; bf16, fp16 or fp32, any strides that are multiples
    of 16 bytes with contiguous channels; an output may be its input.  positions: int64 [B, T] or
    None (the token's index).  inv_freq: fp32 [rotary_dim / 2] or None (no rotation).  q_weight, k_weight:
    fp32 [D] or None.  norm: "rms", "l2" or None.  interleaved: pairs (2i, 2i + 1) instead of
    (i, i + rotary_dim / 2).
    """
    B, T, Hq, Hk, D, R, code = _check(q, k, positions, inv_freq, norm, q_weight, k_weight, q_out, k_out)
    index = _gpu_index(q)
    with _On(index):
        st = lib().kda_qk_rope(q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), _ptr(q_weight),
                               _ptr(k_weight), _ptr(inv_freq) if R else None, _ptr(positions), B, T, Hq, Hk, D, R, code,
                               NORMS[norm], float(eps), bool(interleaved), float(attention_factor),
                               _row_strides(q, k, q_out, k_out), _raw_stream(stream, index))
    if st != KDA_OK:
        raise KDAError(st, "kda_qk_rope")


def bwd(q, k, positions, inv_freq, dq_out, dk_out, *, q_weight=None, k_weight=None, norm="rms", eps=1e-6,
        interleaved=False, attention_factor=1.0, workspace=None, stream=None):
    """Gradients of ``fwd`` from its inputs and dq_out, dk_out (of q's and k's shape and dtype).  Returns a dict: dq, dk
    (contiguous, of q's dtype) and, for the weights given, dq_weight, dk_weight (fp32 [D]).  stream: as in ``linattn.fwd``."""
    B, T, Hq, Hk, D, R, code = _check(q, k, positions, inv_freq, norm, q_weight, k_weight, dq_out, dk_out)
    index = _gpu_index(q)
    L = lib()
    with _On(index):
        with _pool(stream):
            r = {"dq": torch.empty(q.shape, dtype=q.dtype, device=index),
                 "dk": torch.empty(k.shape, dtype=q.dtype, device=index)}
            if q_weight is not None:
                r["dq_weight"] = torch.empty(D, dtype=torch.float32, device=index)
            if k_weight is not None:
                r["dk_weight"] = torch.empty(D, dtype=torch.float32, device=index)
        _used_here(stream, index, *r.values())
        need = L.kda_qk_rope_bwd_workspace_size(B, T, Hq, Hk, D) if len(r) > 2 else 0
        workspace = _workspace(workspace, need, index, stream)
        st = L.kda_qk_rope_bwd(q.data_ptr(), k.data_ptr(), dq_out.data_ptr(), dk_out.data_ptr(), r["dq"].data_ptr(),
                               r["dk"].data_ptr(), _ptr(q_weight), _ptr(k_weight), _ptr(r.get("dq_weight")),
                               _ptr(r.get("dk_weight")), _ptr(inv_freq) if R else None, _ptr(positions), B, T, Hq, Hk, D,
                               R, code, NORMS[norm], float(eps), bool(interleaved), float(attention_factor),
                               _row_strides(q, k, dq_out, dk_out, r["dq"], r["dk"]), _ptr(workspace),
                               _bytes(workspace), _raw_stream(stream, index))
    if st != KDA_OK:
        raise KDAError(st, "kda_qk_rope_bwd")
    return r
