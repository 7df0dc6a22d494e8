"""gated_delta_rule_86_amd -- Kimi Delta Attention (KDA) chunked forward pass for MI355X (gfx950),
with the operators that stand next to it.

The compute path is libkda.so (hand-written HIP kernels behind the C ABI in include/kda.h);
``kda.fwd`` is its thin Python binding.  ``linattn`` is linear attention with a decay for each
head, ``qkrope`` the normalisation and position rotation of queries and keys.  ``workloads``
draws the seeded synthetic inputs.
"""
from . import kda, linattn, qkrope
from .kda import KDAError, fwd, workspace_size

__all__ = ["kda", "linattn", "qkrope", "fwd", "workspace_size", "KDAError"]
