"""The gated delta rule with a decay for each head: kda_gdn_fwd and kda_gdn_fwd_recurrent of libkda.so (include/kda.h).

    S~ = e^{g_t} S_{t-1},   S_t = S~ + beta_t (v_t - S~ k_t) k_t^T,   out_t = scale * S_t q_t

per sequence and head, with the state layout, sequence lengths and calling manner of ``kda`` and ``linattn``.
``qkrope.fwd(..., norm="l2")`` makes the keys of norm 1 that the rule wants.  Argument marshalling only; there is no
fallback path.
"""
from __future__ import annotations

import torch

from . import kda
from .kda import KDA_OK, KDAError, _ptr, lib
from .linattn import _bytes, _check_inputs, _check_state, _code, _gpu_index, _On, _raw_stream, _row_strides, _workspace

D = 128


def workspace_size(B: int, T: int, H: int, N: int = 0, varlen: bool = False) -> int:
    return int(lib().kda_gdn_fwd_workspace_size(B, T, H, N, 1 if varlen else 0))


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


device_status = kda.device_status
