"""Plain 64-bit references of the decayed linear attention and of the q/k norm with position rotation, and the
tolerances that their tests use.

Tolerances count roundings.  A bf16 output is rounded once, by at most 2^-8 of its value; everything before it
is fp32 or better, so the outputs' rel L2 error stays below 2^-8, and an element is off by at most
2^-8 of its value plus the fp32 work on its terms (FP32_SUM times the root mean square).  fp32 outputs are sums
of up to some thousand products with 24-bit factors, each rounded to fp32 (2^-24): errors grow with the root
of the count in the norm and at most linearly in one element.
"""
import math

import torch

D = 128
BF16_STEP = 2.0 ** -8
FP32_REL_L2 = 1e-5     # 2^-24 * sqrt(2^14) < 8e-6: 128 channels x 128 tokens of terms, errors independent
FP32_MAX = 1e-4        # one element against the rms: the same sum with errors five times the rms


def dev():
    return torch.device("cuda:0")


def lin_ref(q, k, v, decay, scale, h0=None, cu=None):
    """Token by token in fp64 on the CPU or GPU the inputs live on; differentiable.  Returns (out, final)."""
    B, T, Hk, _ = q.shape
    H = v.shape[2]
    rep = H // Hk
    q, k, v = q.double().repeat_interleave(rep, 2), k.double().repeat_interleave(rep, 2), v.double()
    g = decay.double().clamp(-1000.0, 0.0).expand(B, T, H)
    bounds = [(b, 0, T) for b in range(B)] if cu is None else [(0, cu[i], cu[i + 1]) for i in range(len(cu) - 1)]
    out, final = [], []
    for n, (b, lo, hi) in enumerate(bounds):
        S = torch.zeros(H, D, D, dtype=torch.float64, device=q.device) if h0 is None else h0[n].double()
        for t in range(lo, hi):
            S = S * g[b, t].exp()[:, None, None] + v[b, t][:, :, None] * k[b, t][:, None, :]
            out.append(scale * (S * q[b, t][:, None, :]).sum(-1))
        final.append(S)
    out = torch.stack(out).reshape(B, T, H, D) if out else q.new_zeros(B, T, H, D)
    return out, torch.stack(final)


def lin_ref_chunked(q, k, v, decay, scale, h0=None, cu=None, C=48):
    """The same in fp64 by chunks of C tokens (another cut than the kernels'), for long sequences; differentiable."""
    B, T, Hk, _ = q.shape
    H = v.shape[2]
    rep = H // Hk
    q, k, v = q.double().repeat_interleave(rep, 2), k.double().repeat_interleave(rep, 2), v.double()
    g = decay.double().clamp(-1000.0, 0.0).expand(B, T, H)
    bounds = [(b, 0, T) for b in range(B)] if cu is None else [(0, cu[i], cu[i + 1]) for i in range(len(cu) - 1)]
    out, final = [], []
    for n, (b, lo, hi) in enumerate(bounds):
        S = torch.zeros(H, D, D, dtype=torch.float64, device=q.device) if h0 is None else h0[n].double()
        for a in range(lo, hi, C):
            e = min(a + C, hi)
            Q, K, V = (x[b, a:e].transpose(0, 1) for x in (q, k, v))
            c = g[b, a:e].t().cumsum(-1)
            low = torch.ones(e - a, e - a, dtype=torch.bool, device=q.device).tril()
            w = torch.where(low, c[:, :, None] - c[:, None, :], -math.inf).exp()
            o = ((Q @ K.mT.contiguous()) * w) @ V + (Q * c.exp()[..., None]) @ S.mT.contiguous()
            out.append((scale * o).transpose(0, 1))
            S = S * c[:, -1].exp()[:, None, None] + (V * (c[:, -1:] - c).exp()[..., None]).mT.contiguous() @ K
        final.append(S)
    out = torch.cat(out).reshape(B, T, H, D) if out else q.new_zeros(B, T, H, D)
    return out, torch.stack(final)


def close_bf16(got, want, what):
    """Rounded once from fp32: half a step of the value (2^-8 relative to it), plus 2^-8 of the rms for what the
    terms' own bf16 hi + lo cuts (2^-17 each) and fp32 sums leave where terms cancel."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape, what
    if not want.numel():
        return
    assert torch.isfinite(got).all(), what
    rms = want.square().mean().sqrt()
    err = (got - want).abs()
    bad = err > BF16_STEP * want.abs() + 2.0 ** -8 * 0.25 * rms
    assert not bad.any(), (what, float(err.max()), float(rms), int(bad.sum()))
    rel = float(err.norm() / want.norm()) if want.norm() > 0 else float(err.norm())
    assert rel <= BF16_STEP, (what, rel)


def close_fp32(got, want, what, rel_l2=FP32_REL_L2, most=FP32_MAX):
    got, want = got.double(), want.double()
    assert got.shape == want.shape, what
    if not want.numel():
        return
    assert torch.isfinite(got).all(), what
    rms = want.square().mean().sqrt()
    err = (got - want).abs()
    if rms == 0:
        assert float(err.max()) == 0.0, what
        return
    rel = float(err.norm() / want.norm())
    assert rel <= rel_l2, (what, rel)
    assert float((err / torch.maximum(rms, want.abs())).max()) <= most, (what, float(err.max()), float(rms))


def inputs(B, T, Hk, H, seed, decay="token", strided=False, lo=1e-3, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
    if strided:
        qkv = n(B, T, (2 * Hk + H) * D + 16).bfloat16()[..., 8:-8]
        q, k, v = qkv.split([Hk * D, Hk * D, H * D], dim=-1)
        q, k, v = (x.unflatten(2, (-1, D)) for x in (q, k, v))
    else:
        q, k, v = n(B, T, Hk, D).bfloat16(), n(B, T, Hk, D).bfloat16(), n(B, T, H, D).bfloat16()
    shape = (B, T, H) if decay == "token" else (H,)
    d = -torch.exp(torch.rand(shape, generator=g, device=device) * -math.log(lo) + math.log(lo))
    return q, k, v, d, n


def close_ddecay(got, want, q, dq, k, dk, decay, final=None, dfinal=None, what="ddecay"):
    """dg_t = sum over the later tokens u of its segment (512 at most) of q_u.dq_u - k_u.dk_u, plus <S, dS> at its end.

    Rounding errors of one product q_u.dq_u against |q_u| |dq_u| / sqrt(128), the size of such a product of
    independent vectors: two exponentials (2^-23 each, one ulp), two chains of 8 to 12 matrix steps (each step rounds
    the running sum, 2^-24: 2^-21 together for each chain), the row product of 32 fused steps and a tree
    (sqrt(35) 2^-24 = 2^-21.4); in all 2^-19.6, and the same for k.dk, independent from token to token.  <S, dS> sums
    16384 products, 64 in a row (2^-21), of states with two such factors (2^-22): 2^-20.4 |S| |dS| / 128.
    A token's error adds up over the n_u <= 512 tokens that see it: in the norm over tokens sqrt(n_u), in a per-head
    decay's sum n_u."""
    B, T, H = q.shape[0], q.shape[1], decay.shape[-1]
    if T == 0:
        assert not got.double().abs().sum() > 0, what
        return
    rep = H // q.shape[2]
    norm = lambda x: x.double().norm(dim=-1)  # noqa: E731
    a = ((norm(q) * norm(dq)) ** 2 + (norm(k) * norm(dk)) ** 2) / D * 2.0 ** -39.2
    a = a.repeat_interleave(rep, 2)                                    # [B, T, H]
    n = torch.arange(1, T + 1, device=q.device).clamp(max=512).double()[None, :, None]
    x = torch.zeros(H, dtype=torch.float64, device=q.device)
    if dfinal is not None:
        x = (final.double().flatten(2).norm(dim=-1) * dfinal.double().flatten(2).norm(dim=-1) * 2.0 ** -20.4 / D).square().sum(0)
    err = (got.double() - want.double())
    most = min(T, 512)
    if decay.dim() == 3:
        tol = float(((a * n).sum() + (x * most).sum()).sqrt())
        assert float(err.norm()) <= tol + 2.0 ** -24 * float(want.norm()), (what, float(err.norm()), tol)
    else:
        tol = ((a * n ** 2).sum((0, 1)) + x * most ** 2).sqrt()
        assert (err.abs() <= 2 * tol + 2.0 ** -24 * want.abs()).all(), (what, err, tol)  # one value: two sigma
