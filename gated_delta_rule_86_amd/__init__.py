"""gated_delta_rule_86_amd -- Kimi Delta Attention (KDA) chunked forward pass for MI355X (gfx950),
with the operators that stand next to it.

The compute path is libkda.so (hand-written HIP kernels behind the C ABI in include/kda.h);
``kda.fwd`` is its thin Python binding.  ``gdn`` is the gated delta rule and ``linattn`` linear
attention, each with a decay for each head, ``qkrope`` the normalisation and position rotation of
queries and keys, ``blocknorm`` the norms after a mixer and before the next block.  ``workloads`` draws the seeded synthetic inputs.
"""
from . import blocknorm, gdn, kda, linattn, qkrope
from .kda import KDAError, fwd, workspace_size

__all__ = ["kda", "blocknorm", "gdn", "linattn", "qkrope", "fwd", "workspace_size", "KDAError"]
