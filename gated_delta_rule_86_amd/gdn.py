"""The gated delta rule with a decay for each head: kda_gdn_fwd, kda_gdn_fwd_recurrent and
kda_gdn_bwd of libkda.so (include/kda.h).

    S~ = e^{g_t} S_{t-1},   S_t = S~ + beta_t (v_t - S~ k_t) k_t^T,   out_t = scale * S_t q_t

per sequence and head, with the state layout, sequence lengths and calling manner of ``kda`` and ``linattn``.
``qkrope.fwd(..., norm="l2")`` makes the keys of norm 1 that the rule wants.  Argument marshalling only; there is no
fallback path.
"""
from __future__ import annotations

import torch

from . import kda
from .kda import KDA_OK, KDAError, _pool, _ptr, _used_here, lib
from .linattn import _bytes, _check_inputs, _check_state, _code, _gpu_index, _On, _raw_stream, _row_strides, _workspace

D = 128


def workspace_size(B: int, T: int, H: int, N: int = 0, varlen: bool = False) -> int:
    return int(lib().kda_gdn_fwd_workspace_size(B, T, H, N, 1 if varlen else 0))


def bwd_workspace_size(B: int, T: int, Hk: int, H: int, N: int = 0, varlen: bool = False) -> int:
    return int(lib().kda_gdn_bwd_workspace_size(B, T, Hk, H, N, 1 if varlen else 0))


def _check(q, k, v, decay, beta, cu_seqlens, cu_seqlens_host):
    if decay.dim() != 3:
        raise ValueError("decay must be a contiguous fp32 [B, T, H] tensor")
    got = _check_inputs(q, k, v, decay, cu_seqlens, cu_seqlens_host)
    if (beta.dtype is not torch.float32 or beta.shape != decay.shape or not beta.is_contiguous()
            or beta.get_device() != q.get_device()):
        raise ValueError("beta must be a contiguous fp32 [B, T, H] tensor on q's device")
    return got


def fwd(q, k, v, decay, beta, scale, out, initial_state=None, final_state=None, cu_seqlens=None, *,
        cu_seqlens_host=None, workspace=None, stream=None, _recurrent=False):
    """Chunked forward pass on torch device tensors; writes ``out`` and ``final_state`` in place and
    returns the workspace.

    q, k: bf16 [B, T, Hk, 128]; v: bf16 [B, T, H, 128], H a multiple of Hk (views with contiguous
    channels and strides that are multiples of 8 are read in place); decay: fp32 [B, T, H], natural-log
    decays <= 0; beta: fp32 [B, T, H], write strengths; out: contiguous bf16 [B, T, H, 128]; states: bf16 or fp32
    [N, H, 128, 128] or None, final_state may be initial_state; cu_seqlens: int64 [N+1] device
    tensor (then B is 1) or None.  cu_seqlens_host, workspace, stream: as in ``linattn.fwd``.
    """
    B, T, Hk, H, N, K, V, _, host = _check(q, k, v, decay, beta, cu_seqlens, cu_seqlens_host)
    if (out.dtype is not torch.bfloat16 or out.shape != v.shape or not out.is_contiguous()
            or out.get_device() != q.get_device()):
        raise ValueError("out must be a contiguous bf16 [B, T, H, 128] tensor on q's device")
    _check_state("initial_state", initial_state, (N, H, V, K), q)
    _check_state("final_state", final_state, (N, H, V, K), q)
    h0_code, ht_code = _code(initial_state), _code(final_state)
    if h0_code and ht_code and h0_code != ht_code:
        raise ValueError("initial_state and final_state dtypes must match")
    index = _gpu_index(q)
    L = lib()
    varlen = cu_seqlens is not None
    if _recurrent:
        need, call = (256 if varlen else 0), L.kda_gdn_fwd_recurrent
    else:
        need, call = L.kda_gdn_fwd_workspace_size(B, T, H, N if varlen else 0, varlen), L.kda_gdn_fwd
    with _On(index):
        if workspace is not None or need:
            workspace = _workspace(workspace, need, index, stream)
        st = call(q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(), beta.data_ptr(), float(scale),
                  out.data_ptr(), _ptr(initial_state), h0_code, _ptr(final_state), ht_code, _ptr(cu_seqlens),
                  None if host is None else host.ctypes.data, B, T, Hk, H, N if varlen else B, K, V,
                  _row_strides(q, k, v), _ptr(workspace), _bytes(workspace), _raw_stream(stream, index))
    if st != KDA_OK:
        raise KDAError(st, "kda_gdn_fwd_recurrent" if _recurrent else "kda_gdn_fwd")
    return workspace


def fwd_recurrent(q, k, v, decay, beta, scale, out, initial_state=None, final_state=None, cu_seqlens=None, **kw):
    """The same operator token by token in fp32: the decode step (one token per sequence, state in and
    out) and other short sequences.  Same arguments and keywords as ``fwd``; without cu_seqlens
    it needs no workspace and returns None."""
    return fwd(q, k, v, decay, beta, scale, out, initial_state, final_state, cu_seqlens, _recurrent=True, **kw)


def bwd(q, k, v, decay, beta, scale, dout, initial_state=None, dfinal_state=None, cu_seqlens=None, *,
        need_dinitial_state=True, cu_seqlens_host=None, workspace=None, stream=None):
    """Gradients of ``fwd``'s out and final_state (kda_gdn_bwd in include/kda.h).

    Inputs as ``fwd``; dout: contiguous bf16 [B, T, H, 128]; dfinal_state: None or fp32
    [N, H, 128, 128].  Returns a dict of device tensors: dq, dk (bf16, shape of q), dv (bf16), ddecay, dbeta
    (fp32 [B, T, H]), dinitial_state (fp32 [N, H, 128, 128]; also without an initial state,
    unless need_dinitial_state is False) and the workspace used.
    """
    B, T, Hk, H, N, K, V, _, host = _check(q, k, v, decay, beta, cu_seqlens, cu_seqlens_host)
    if (dout.dtype is not torch.bfloat16 or dout.shape != v.shape or not dout.is_contiguous()
            or dout.get_device() != q.get_device()):
        raise ValueError("dout must be a contiguous bf16 [B, T, H, 128] tensor on q's device")
    _check_state("initial_state", initial_state, (N, H, V, K), q)
    _check_state("dfinal_state", dfinal_state, (N, H, V, K), q, bf16_too=False)
    index = _gpu_index(q)
    varlen = cu_seqlens is not None
    L = lib()
    need = L.kda_gdn_bwd_workspace_size(B, T, Hk, H, N if varlen else 0, varlen)
    with _On(index):
        bf16, fp32 = torch.bfloat16, torch.float32
        with _pool(stream):
            r = {"dq": torch.empty((B, T, Hk, K), dtype=bf16, device=index),
                 "dk": torch.empty((B, T, Hk, K), dtype=bf16, device=index),
                 "dv": torch.empty((B, T, H, V), dtype=bf16, device=index),
                 "ddecay": torch.empty((B, T, H), dtype=fp32, device=index),
                 "dbeta": torch.empty((B, T, H), dtype=fp32, device=index)}
            if need_dinitial_state:
                r["dinitial_state"] = torch.empty((N, H, V, K), dtype=fp32, device=index)
        _used_here(stream, index, *r.values())
        workspace = _workspace(workspace, need or 1, index, stream)
        st = L.kda_gdn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(), beta.data_ptr(), float(scale),
                           _ptr(initial_state), _code(initial_state), dout.data_ptr(), _ptr(dfinal_state),
                           r["dq"].data_ptr(), r["dk"].data_ptr(), r["dv"].data_ptr(), r["ddecay"].data_ptr(),
                           r["dbeta"].data_ptr(), _ptr(r.get("dinitial_state")), _ptr(cu_seqlens),
                           None if host is None else host.ctypes.data, B, T, Hk, H, N if varlen else B, K, V,
                           _row_strides(q, k, v), workspace.data_ptr(), _bytes(workspace), _raw_stream(stream, index))
    if st != KDA_OK:
        raise KDAError(st, "kda_gdn_bwd")
    r["workspace"] = workspace
    return r


device_status = kda.device_status
