"""Linear attention with a decay for each head: kda_lin_fwd, kda_lin_fwd_recurrent and
kda_lin_bwd of libkda.so (include/kda.h).

    S_t = e^{g_t} S_{t-1} + v_t k_t^T,     out_t = scale * S_t q_t

per sequence and head, with the state layout, sequence lengths and calling manner of ``kda``.
Argument marshalling only; there is no fallback path.
"""
from __future__ import annotations

import ctypes

from . import kda
from .kda import KDA_OK, KDAError, _ptr, _state_code, _stream_handle, lib

D = 128


def workspace_size(B: int, T: int, H: int, N: int = 0, varlen: bool = False) -> int:
    return int(lib().kda_lin_fwd_workspace_size(B, T, H, N, 1 if varlen else 0))


def bwd_workspace_size(B: int, T: int, Hk: int, H: int, N: int = 0, varlen: bool = False,
                       need_ddecay: bool = True) -> int:
    return int(lib().kda_lin_bwd_workspace_size(B, T, Hk, H, N, 1 if varlen else 0, 1 if need_ddecay else 0))


def _row_strides(*tensors):
    """Batch, token and head strides in elements, or None when every tensor is contiguous.  The
    stride of a dimension of size 1 is never used and taken as 0."""
    if all(t.is_contiguous() for t in tensors):
        return None
    got = []
    for t in tensors:
        got += [0 if n == 1 else s for n, s in zip(t.shape[:3], t.stride()[:3])]
    return (ctypes.c_int64 * len(got))(*got)


def _check_inputs(q, k, v, decay, cu_seqlens, cu_seqlens_host):
    import torch
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v must be [B, T, heads, 128]")
    B, T, Hk, K = q.shape
    H, V = v.shape[2], v.shape[3]
    if tuple(k.shape) != (B, T, Hk, K) or tuple(v.shape[:2]) != (B, T):
        raise ValueError("q and k must be [B, T, Hk, 128], v [B, T, H, 128]")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or (t.stride(3) != 1 and t.shape[3] != 1):
            raise ValueError(f"{name} must be bf16 with contiguous channels")
    if decay.dtype != torch.float32 or not decay.is_contiguous() or tuple(decay.shape) not in ((H,), (B, T, H)):
        raise ValueError("decay must be a contiguous fp32 [H] or [B, T, H] tensor")
    N = B
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int64 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be a contiguous int64 [N+1] tensor")
        N = cu_seqlens.numel() - 1
    for name, t in (("k", k), ("v", v), ("decay", decay), ("cu_seqlens", cu_seqlens)):
        if t is not None and t.device != q.device:
            raise ValueError(f"{name} must be on q's device")
    host = None
    if cu_seqlens_host is not None:
        import numpy as np
        host = np.ascontiguousarray(np.asarray(cu_seqlens_host, dtype=np.int64))
        if cu_seqlens is None or host.shape != (N + 1,):
            raise ValueError("cu_seqlens_host must be the host copy of cu_seqlens")
    return B, T, Hk, H, N, K, V, decay.dim() == 3, host


def _check_state(name, t, shape, device, dtypes):
    if t is not None and (tuple(t.shape) != shape or not t.is_contiguous() or t.dtype not in dtypes
                          or t.device != device):
        raise ValueError(f"{name} must be a contiguous {list(shape)} tensor of {' or '.join(map(str, dtypes))} "
                         "on q's device")


def _workspace(workspace, need, device, stream):
    import torch
    if workspace is not None:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on q's device")
        return workspace
    if need == 0:
        return None
    workspace = torch.empty(need, dtype=torch.uint8, device=device)
    # allocated on the current stream; the kernels run on `stream`: keep the caching
    # allocator from reusing the block before they have finished
    if stream is not None and stream != torch.cuda.current_stream(device):
        workspace.record_stream(stream)
    return workspace


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def fwd(q, k, v, decay, scale, out, initial_state=None, final_state=None, cu_seqlens=None, *,
        cu_seqlens_host=None, workspace=None, stream=None, _recurrent=False):
    """Chunked forward pass on torch device tensors; writes ``out`` and ``final_state`` in place and
    returns the workspace.

    q, k: bf16 [B, T, Hk, 128]; v: bf16 [B, T, H, 128], H a multiple of Hk (views with contiguous
    channels and strides that are multiples of 8 are read in place); decay: fp32 natural-log
    decays <= 0, [H] or [B, T, H]; out: contiguous bf16 [B, T, H, 128]; states: bf16 or fp32
    [N, H, 128, 128] or None, final_state may be initial_state; cu_seqlens: int64 [N+1] device
    tensor (then B is 1) or None.  cu_seqlens_host, workspace, stream: as in ``kda.fwd``.
    """
    import torch
    B, T, Hk, H, N, K, V, per_token, host = _check_inputs(q, k, v, decay, cu_seqlens, cu_seqlens_host)
    if out.dtype != torch.bfloat16 or out.shape != v.shape or not out.is_contiguous() or out.device != q.device:
        raise ValueError("out must be a contiguous bf16 [B, T, H, 128] tensor on q's device")
    kinds = (torch.bfloat16, torch.float32)
    _check_state("initial_state", initial_state, (N, H, V, K), q.device, kinds)
    _check_state("final_state", final_state, (N, H, V, K), q.device, kinds)
    if initial_state is not None and final_state is not None and initial_state.dtype != final_state.dtype:
        raise ValueError("initial_state and final_state dtypes must match")
    varlen = cu_seqlens is not None
    need = (256 if varlen else 0) if _recurrent else workspace_size(B, T, H, N if varlen else 0, varlen)
    call = lib().kda_lin_fwd_recurrent if _recurrent else lib().kda_lin_fwd
    with torch.cuda.device(q.device):
        workspace = _workspace(workspace, need, q.device, stream)
        st = call(_ptr(q), _ptr(k), _ptr(v), _ptr(decay), int(per_token), float(scale), _ptr(out),
                  _ptr(initial_state), _state_code(initial_state), _ptr(final_state), _state_code(final_state),
                  _ptr(cu_seqlens), None if host is None else host.ctypes.data, B, T, Hk, H, N if varlen else B, K, V,
                  _row_strides(q, k, v), _ptr(workspace), _bytes(workspace), _stream_handle(stream, q.device))
    if st != KDA_OK:
        raise KDAError(st, "kda_lin_fwd_recurrent" if _recurrent else "kda_lin_fwd")
    return workspace


def fwd_recurrent(q, k, v, decay, scale, out, initial_state=None, final_state=None, cu_seqlens=None, **kw):
    """The same operator token by token in fp32: the decode step (one token per sequence, state in and
    out) and other short sequences.  Same arguments and keywords as ``fwd``; without cu_seqlens
    it needs no workspace and returns None."""
    return fwd(q, k, v, decay, scale, out, initial_state, final_state, cu_seqlens, _recurrent=True, **kw)


def bwd(q, k, v, decay, scale, dout, initial_state=None, dfinal_state=None, cu_seqlens=None, *, need_ddecay=True,
        cu_seqlens_host=None, workspace=None, stream=None):
    """Gradients of ``fwd``'s out and final_state (kda_lin_bwd in include/kda.h).

    Inputs as ``fwd``; dout: contiguous bf16 [B, T, H, 128]; dfinal_state: None or fp32
    [N, H, 128, 128].  Returns a dict of device tensors: dq, dk (bf16, shape of q), dv (bf16), ddecay
    (fp32, shape of decay; with need_ddecay), dinitial_state (fp32 [N, H, 128, 128]) and the
    workspace used.
    """
    import torch
    B, T, Hk, H, N, K, V, per_token, host = _check_inputs(q, k, v, decay, cu_seqlens, cu_seqlens_host)
    dev = q.device
    if dout.dtype != torch.bfloat16 or dout.shape != v.shape or not dout.is_contiguous() or dout.device != dev:
        raise ValueError("dout must be a contiguous bf16 [B, T, H, 128] tensor on q's device")
    _check_state("initial_state", initial_state, (N, H, V, K), dev, (torch.bfloat16, torch.float32))
    _check_state("dfinal_state", dfinal_state, (N, H, V, K), dev, (torch.float32,))
    varlen = cu_seqlens is not None
    need = bwd_workspace_size(B, T, Hk, H, N if varlen else 0, varlen, need_ddecay)
    with torch.cuda.device(dev):
        empty = lambda shape, dt: torch.empty(shape, dtype=dt, device=dev)  # noqa: E731
        r = {"dq": empty((B, T, Hk, K), torch.bfloat16), "dk": empty((B, T, Hk, K), torch.bfloat16),
             "dv": empty((B, T, H, V), torch.bfloat16), "dinitial_state": empty((N, H, V, K), torch.float32)}
        if need_ddecay:
            r["ddecay"] = empty(tuple(decay.shape), torch.float32)
        if stream is not None and stream != torch.cuda.current_stream(dev):
            for t in r.values():
                t.record_stream(stream)
        workspace = _workspace(workspace, max(need, 1), dev, stream)
        st = lib().kda_lin_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(decay), int(per_token), float(scale),
                               _ptr(initial_state), _state_code(initial_state), _ptr(dout), _ptr(dfinal_state),
                               _ptr(r["dq"]), _ptr(r["dk"]), _ptr(r["dv"]), _ptr(r.get("ddecay")),
                               _ptr(r["dinitial_state"]), _ptr(cu_seqlens),
                               None if host is None else host.ctypes.data, B, T, Hk, H, N if varlen else B, K, V,
                               _row_strides(q, k, v), _ptr(workspace), _bytes(workspace),
                               _stream_handle(stream, dev))
    if st != KDA_OK:
        raise KDAError(st, "kda_lin_bwd")
    r["workspace"] = workspace
    return r


device_status = kda.device_status
