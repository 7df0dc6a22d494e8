"""How far the decays' gradients of the gated delta rule may be off, token by token.

dg_t = <dS~_t, S~_t> is the inner product of what comes to token t from before and of what its state is read for from t on.  In a
block of 64 tokens, with S the state before it and dS the gradient behind it, the two are sums of
    e^{b_t} S,  e^{b_t - b_s} w_s k_s^T (s < t)        and        e^{L - b_t} dS,  e^{b_u - b_t} (scale dO_u q_u^T - dx_u k_u^T) (u >= t).
Their sizes, the terms taken as independent, are the roots of the sums of their squares, A_t and C_t.  Each term is the product of
vectors that are off by FP32_REL_L2 (derived in gdn_testutil; the chunks of 32 tokens that the kernels use have shorter chains than
the 64 counted there) of their size in independent directions: a dot product with such a vector of 128 values is off by
FP32_REL_L2 / sqrt(128) of the sizes.  So dg_t is off by FP32_REL_L2 A_t C_t / sqrt(128) in the norm, one value by up to four times
that, and by the decay factors' own error: the exponential of a 24-bit difference x is off by 2^-25 |x| ln 2 twice (the difference
and its rounding), below 2^-24 |g| of the value.  All of it is scaled by e^{g_t}, however small."""
import torch

from gdn_testutil import D, FP32_REL_L2

BLOCK = 64


def crossing_size(q, k, v, decay, beta, scale, dout, h0=None, dht=None, cu=None):
    """A_t C_t of each token, [B, T, H] in fp64, and the largest one without the token's own decay."""
    B, T, Hk, _ = q.shape
    H = v.shape[2]
    rep = H // Hk
    q, k, v = q.double().repeat_interleave(rep, 2), k.double().repeat_interleave(rep, 2), v.double()
    beta, do = beta.double(), dout.double() * scale
    a = decay.double().clamp(-1000.0, 0.0).exp()
    bounds = [(b, 0, T) for b in range(B)] if cu is None else [(0, cu[i], cu[i + 1]) for i in range(len(cu) - 1)]
    came, before, read = (torch.zeros_like(a) for _ in range(3))
    size = lambda x: x.flatten(1).norm(dim=1)  # noqa: E731
    for n, (b, lo, hi) in enumerate(bounds):
        S = torch.zeros(H, D, D, dtype=torch.float64, device=q.device) if h0 is None else h0[n].double()
        A = size(S)
        for t in range(lo, hi):
            if (t - lo) % BLOCK == 0:
                A = size(S)
            before[b, t], A = A, A * a[b, t]
            came[b, t] = A
            S = S * a[b, t][:, None, None]
            w = (v[b, t] - (S * k[b, t][:, None, :]).sum(-1)) * beta[b, t][:, None]
            S = S + w[:, :, None] * k[b, t][:, None, :]
            A = (A.square() + (w.norm(dim=1) * k[b, t].norm(dim=1)).square()).sqrt()
        dS = torch.zeros_like(S) if dht is None else dht[n].double()
        for t in reversed(range(lo, hi)):
            if t == hi - 1 or (t - lo) % BLOCK == BLOCK - 1:
                C = size(dS)
            dS = dS + do[b, t][:, :, None] * q[b, t][:, None, :]
            dx = (dS * k[b, t][:, None, :]).sum(-1) * beta[b, t][:, None]
            dS = dS - dx[:, :, None] * k[b, t][:, None, :]
            C = (C.square() + (do[b, t].norm(dim=1) * q[b, t].norm(dim=1)).square()
                 + (dx.norm(dim=1) * k[b, t].norm(dim=1)).square()).sqrt()
            read[b, t] = C
            C, dS = C * a[b, t], dS * a[b, t][:, None, None]
    return came * read, float((before * read).amax()) if T else 0.0


def ddecay_is_close(got, want, size, decay, what="", grow=1.0):
    """Raises where ddecay is off by more than the bounds above, times grow, and what factors below 2^-126, the smallest normal fp32
    number, leave: they count as 0, in each of a block's terms.  size: what crossing_size returns."""
    gone = 2.0 ** -126 * BLOCK * size[1]
    got, size = got.double(), grow * FP32_REL_L2 / D ** 0.5 * size[0]
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    if not got.numel():
        return
    err = (got - want).abs()
    own = 2.0 ** -24 * (1.0 - decay.double().clamp(-1000.0, 0.0)) * want.abs()
    bad = err > 4 * size + own + gone
    assert not bad.any(), (what, int(bad.sum()), float((err / (4 * size + own + gone)).max()))
    assert float(err.norm()) <= float(size.norm()) + float(own.norm()) + float(gone), (what, float(err.norm()), float(size.norm()))
