"""Linear attention with a decay for each head: kda_lin_fwd, kda_lin_fwd_recurrent and
kda_lin_bwd of libkda.so (include/kda.h).

    S_t = e^{g_t} S_{t-1} + v_t k_t^T,     out_t = scale * S_t q_t

per sequence and head, with the state layout, sequence lengths and calling manner of ``kda``.
Argument marshalling only; there is no fallback path.
"""
from __future__ import annotations

import ctypes

import torch

from . import kda
from .kda import KDA_OK, KDAError, _pool, _ptr, _used_here, lib

D = 128


def workspace_size(B: int, T: int, H: int, N: int = 0, varlen: bool = False) -> int:
    return int(lib().kda_lin_fwd_workspace_size(B, T, H, N, 1 if varlen else 0))


def bwd_workspace_size(B: int, T: int, Hk: int, H: int, N: int = 0, varlen: bool = False,
                       need_ddecay: bool = True) -> int:
    return int(lib().kda_lin_bwd_workspace_size(B, T, Hk, H, N, 1 if varlen else 0, 1 if need_ddecay else 0))


def _row_strides(*tensors):
    """Batch, token and head strides in elements, or None when every tensor is contiguous.  The
    stride of a dimension of size 1 is never used and taken as 0."""
    for t in tensors:
        if not t.is_contiguous():
            break
    else:
        return None
    got = []
    for t in tensors:
        s, n = t.stride(), t.shape
        got += (s[0] if n[0] > 1 else 0, s[1] if n[1] > 1 else 0, s[2] if n[2] > 1 else 0)
    return (ctypes.c_int64 * len(got))(*got)


def _gpu_index(t):
    i = t.get_device()
    if i < 0:
        raise ValueError("tensors must be on a GPU")
    return i


class _On:
    """The call runs with q's device current; only a change costs anything."""

    __slots__ = ("guard",)

    def __init__(self, index):
        self.guard = None if torch.cuda.current_device() == index else torch.cuda.device(index)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *e):
        if self.guard is not None:
            self.guard.__exit__(*e)


def _raw_stream(stream, index):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if stream.device.index != index:
        raise ValueError(f"stream must be on the tensors' device, cuda:{index}, not on {stream.device}")
    return stream.cuda_stream


def _check_inputs(q, k, v, decay, cu_seqlens, cu_seqlens_host):
    qs, vs = q.shape, v.shape
    if len(qs) != 4 or len(vs) != 4:
        raise ValueError("q, k and v must be [B, T, heads, 128]")
    B, T, Hk, K = qs
    H, V = vs[2], vs[3]
    if k.shape != qs or vs[0] != B or vs[1] != T:
        raise ValueError("q and k must be [B, T, Hk, 128], v [B, T, H, 128]")
    for t in (q, k, v):
        if t.dtype is not torch.bfloat16 or (t.stride(3) != 1 and t.shape[3] != 1):
            raise ValueError("q, k and v must be bf16 with contiguous channels")
    per_token = decay.dim() == 3
    if decay.dtype is not torch.float32 or not decay.is_contiguous() or decay.shape != ((B, T, H) if per_token else (H,)):
        raise ValueError("decay must be a contiguous fp32 [H] or [B, T, H] tensor")
    N = B
    at = q.get_device()
    if k.get_device() != at or v.get_device() != at or decay.get_device() != at:
        raise ValueError("k, v and decay must be on q's device")
    if cu_seqlens is not None:
        if cu_seqlens.dtype is not torch.int64 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be a contiguous int64 [N+1] tensor")
        if cu_seqlens.get_device() != at:
            raise ValueError("cu_seqlens must be on q's device")
        N = cu_seqlens.numel() - 1
    host = None
    if cu_seqlens_host is not None:
        import numpy as np
        host = np.ascontiguousarray(np.asarray(cu_seqlens_host, dtype=np.int64))
        if cu_seqlens is None or host.shape != (N + 1,):
            raise ValueError("cu_seqlens_host must be the host copy of cu_seqlens")
    return B, T, Hk, H, N, K, V, per_token, host


def _check_state(name, t, shape, q, bf16_too=True):
    if t is not None and (t.shape != shape or not t.is_contiguous() or t.get_device() != q.get_device() or not (
            t.dtype is torch.float32 or (bf16_too and t.dtype is torch.bfloat16))):
        raise ValueError(f"{name} must be a contiguous {list(shape)} tensor of fp32{' or bf16' if bf16_too else ''} "
                         "on q's device")


def _workspace(workspace, need, index, stream):
    if workspace is not None:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on q's device")
        return workspace
    if need == 0:
        return None
    with _pool(stream):
        workspace = torch.empty(need, dtype=torch.uint8, device=index)
    _used_here(stream, index, workspace)
    return workspace


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _code(t):
    return 0 if t is None else 2 if t.dtype is torch.float32 else 1


def fwd(q, k, v, decay, scale, out, initial_state=None, final_state=None, cu_seqlens=None, *,
        cu_seqlens_host=None, workspace=None, stream=None, _recurrent=False):
    """Chunked forward pass on torch device tensors; writes ``out`` and ``final_state`` in place and
    returns the workspace.

    q, k: bf16 [B, T, Hk, 128]; v: bf16 [B, T, H, 128], H a multiple of Hk (views with contiguous
    channels and strides that are multiples of 8 are read in place); decay: fp32 natural-log
    decays <= 0, [H] or [B, T, H]; out: contiguous bf16 [B, T, H, 128]; states: bf16 or fp32
    [N, H, 128, 128] or None, final_state may be initial_state; cu_seqlens: int64 [N+1] device
    tensor (then B is 1) or None.  cu_seqlens_host, workspace, stream: as in ``kda.fwd``.

    With ``stream`` the kernels run there and what the call allocates comes from that stream's pool; the caller orders
    the inputs' producers before it and the results' users behind it, and keeps the tensors it passes alive until then.
    """
    B, T, Hk, H, N, K, V, per_token, host = _check_inputs(q, k, v, decay, cu_seqlens, cu_seqlens_host)
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
        need, call = (256 if varlen else 0), L.kda_lin_fwd_recurrent
    else:
        need, call = L.kda_lin_fwd_workspace_size(B, T, H, N if varlen else 0, varlen), L.kda_lin_fwd
    with _On(index):
        if workspace is not None or need:
            workspace = _workspace(workspace, need, index, stream)
        st = call(q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(), per_token, float(scale), out.data_ptr(),
                  _ptr(initial_state), h0_code, _ptr(final_state), ht_code, _ptr(cu_seqlens),
                  None if host is None else host.ctypes.data, B, T, Hk, H, N if varlen else B, K, V,
                  _row_strides(q, k, v), _ptr(workspace), _bytes(workspace), _raw_stream(stream, index))
    if st != KDA_OK:
        raise KDAError(st, "kda_lin_fwd_recurrent" if _recurrent else "kda_lin_fwd")
    return workspace


def fwd_recurrent(q, k, v, decay, scale, out, initial_state=None, final_state=None, cu_seqlens=None, **kw):
    """The same operator token by token in fp32: the decode step (one token per sequence, state in and
    out) and other short sequences.  Same arguments and keywords as ``fwd``; without cu_seqlens
    it needs no workspace and returns None."""
    return fwd(q, k, v, decay, scale, out, initial_state, final_state, cu_seqlens, _recurrent=True, **kw)


def bwd(q, k, v, decay, scale, dout, initial_state=None, dfinal_state=None, cu_seqlens=None, *, need_ddecay=True,
        need_dinitial_state=True, cu_seqlens_host=None, workspace=None, stream=None):
    """Gradients of ``fwd``'s out and final_state (kda_lin_bwd in include/kda.h).

    Inputs as ``fwd``; dout: contiguous bf16 [B, T, H, 128]; dfinal_state: None or fp32
    [N, H, 128, 128].  Returns a dict of device tensors: dq, dk (bf16, shape of q), dv (bf16), ddecay
    (fp32, shape of decay; with need_ddecay), dinitial_state (fp32 [N, H, 128, 128]; also without an initial state,
    unless need_dinitial_state is False: 64 KiB per sequence and head) and the workspace used.
    """
    B, T, Hk, H, N, K, V, per_token, host = _check_inputs(q, k, v, decay, cu_seqlens, cu_seqlens_host)
    if (dout.dtype is not torch.bfloat16 or dout.shape != v.shape or not dout.is_contiguous()
            or dout.get_device() != q.get_device()):
        raise ValueError("dout must be a contiguous bf16 [B, T, H, 128] tensor on q's device")
    _check_state("initial_state", initial_state, (N, H, V, K), q)
    _check_state("dfinal_state", dfinal_state, (N, H, V, K), q, bf16_too=False)
    index = _gpu_index(q)
    varlen = cu_seqlens is not None
    L = lib()
    need = L.kda_lin_bwd_workspace_size(B, T, Hk, H, N if varlen else 0, varlen, bool(need_ddecay))
    with _On(index):
        bf16, fp32 = torch.bfloat16, torch.float32
        with _pool(stream):
            r = {"dq": torch.empty((B, T, Hk, K), dtype=bf16, device=index),
                 "dk": torch.empty((B, T, Hk, K), dtype=bf16, device=index),
                 "dv": torch.empty((B, T, H, V), dtype=bf16, device=index)}
            if need_dinitial_state:
                r["dinitial_state"] = torch.empty((N, H, V, K), dtype=fp32, device=index)
            if need_ddecay:
                r["ddecay"] = torch.empty(decay.shape, dtype=fp32, device=index)
        _used_here(stream, index, *r.values())
        workspace = _workspace(workspace, need or 1, index, stream)
        st = L.kda_lin_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(), per_token, float(scale),
                           _ptr(initial_state), _code(initial_state), dout.data_ptr(), _ptr(dfinal_state),
                           r["dq"].data_ptr(), r["dk"].data_ptr(), r["dv"].data_ptr(), _ptr(r.get("ddecay")),
                           _ptr(r.get("dinitial_state")), _ptr(cu_seqlens),
                           None if host is None else host.ctypes.data, B, T, Hk, H, N if varlen else B, K, V,
                           _row_strides(q, k, v), workspace.data_ptr(), _bytes(workspace), _raw_stream(stream, index))
    if st != KDA_OK:
        raise KDAError(st, "kda_lin_bwd")
    r["workspace"] = workspace
    return r


device_status = kda.device_status
