"""Plain 64-bit reference of the gated delta rule, and the tolerances that its tests use.

Tolerances count roundings.  A bf16 output is rounded once, by at most 2^-8 of its value; what happens before
is fp32 on factors of 24 bits.  An fp32 output is the end of a chain: per chunk of 64 tokens three products in a row
(state times keys, the triangular system, the state's update), each some 12 matrix steps that round the running sum by 2^-24:
sqrt(36) 2^-24 = 3.6e-7 of the value for independent errors.  Chunks add up like a walk that the decays and the delta rule
damp, at most the root of their count: 10 chunks make 1.1e-6; correlated keys (a triangular system with large
entries) add a small factor, taken as 4: 5e-6 in the norm.  One element of thousands is off by up to ten times the norm's share.
"""
import torch

D = 128
BF16_STEP = 2.0 ** -8
FP32_REL_L2 = 5e-6
FP32_MAX = 5e-5


def gdn_ref(q, k, v, decay, beta, scale, h0=None, cu=None):
    """Token by token in fp64 on the device the inputs live on; differentiable.  Returns (out, final)."""
    B, T, Hk, _ = q.shape
    H = v.shape[2]
    rep = H // Hk
    q, k, v = q.double().repeat_interleave(rep, 2), k.double().repeat_interleave(rep, 2), v.double()
    a, beta = decay.double().clamp(-1000.0, 0.0).exp(), beta.double()
    bounds = [(b, 0, T) for b in range(B)] if cu is None else [(0, cu[i], cu[i + 1]) for i in range(len(cu) - 1)]
    out, final = [], []
    for n, (b, lo, hi) in enumerate(bounds):
        S = torch.zeros(H, D, D, dtype=torch.float64, device=q.device) if h0 is None else h0[n].double()
        for t in range(lo, hi):
            S = S * a[b, t][:, None, None]
            u = (v[b, t] - (S * k[b, t][:, None, :]).sum(-1)) * beta[b, t][:, None]
            S = S + u[:, :, None] * k[b, t][:, None, :]
            out.append(scale * (S * q[b, t][:, None, :]).sum(-1))
        final.append(S)
    out = torch.stack(out).reshape(B, T, H, D) if out else v.new_zeros(B, T, H, D)
    return out, torch.stack(final)


def gdn_ref_bwd(q, k, v, decay, beta, scale, dout, h0=None, dht=None, cu=None):
    """Gradients by the recurrence run backwards in fp64.  Returns a dict with dq, dk, dv, ddecay, dbeta, dinitial_state and the
    sizes of what ddecay and dbeta are sums of: sum_size [B, T, H] (products of q.dq and v.dv), state_size (<S, dS> after the
    token) and beta_size, each for independent vectors (norms multiplied, over the root of the count)."""
    B, T, Hk, _ = q.shape
    H = v.shape[2]
    rep = H // Hk
    q, k, v = q.double().repeat_interleave(rep, 2), k.double().repeat_interleave(rep, 2), v.double()
    g, beta, do = decay.double(), beta.double(), dout.double() * scale
    a = g.clamp(-1000.0, 0.0).exp()
    bounds = [(b, 0, T) for b in range(B)] if cu is None else [(0, cu[i], cu[i + 1]) for i in range(len(cu) - 1)]
    dq, dk, dv = torch.zeros_like(v), torch.zeros_like(v), torch.zeros_like(v)
    dg, db, state_size, beta_size = (torch.zeros_like(a) for _ in range(4))
    dh0 = torch.zeros(len(bounds), H, D, D, dtype=torch.float64, device=q.device)
    for n, (b, lo, hi) in enumerate(bounds):
        S = torch.zeros(H, D, D, dtype=torch.float64, device=q.device) if h0 is None else h0[n].double()
        steps = []
        for t in range(lo, hi):
            decayed = S * a[b, t][:, None, None]
            r = v[b, t] - (decayed * k[b, t][:, None, :]).sum(-1)
            S = decayed + (r * beta[b, t][:, None])[:, :, None] * k[b, t][:, None, :]
            steps.append((t, S, decayed, r))
        dS = torch.zeros_like(S) if dht is None else dht[n].double()
        for t, S, decayed, r in reversed(steps):
            state_size[b, t] = S.flatten(1).norm(dim=1) * dS.flatten(1).norm(dim=1) / D
            dq[b, t] = (S * do[b, t][:, :, None]).sum(1)
            dS = dS + do[b, t][:, :, None] * q[b, t][:, None, :]
            w = (dS * k[b, t][:, None, :]).sum(-1)
            db[b, t] = (w * r).sum(-1)
            beta_size[b, t] = w.norm(dim=1) * r.norm(dim=1) / D ** 0.5
            dr = w * beta[b, t][:, None]
            dv[b, t] = dr
            dk[b, t] = (dS * (r * beta[b, t][:, None])[:, :, None]).sum(1) - (decayed * dr[:, :, None]).sum(1)
            dS = dS - dr[:, :, None] * k[b, t][:, None, :]
            dg[b, t] = (dS * decayed).sum((-1, -2))
            dS = dS * a[b, t][:, None, None]
        dh0[n] = dS
    dg = torch.where((g > -1000.0) & (g <= 0.0), dg, 0.0)
    sum_size = (q.norm(dim=-1) * dq.norm(dim=-1) + v.norm(dim=-1) * dv.norm(dim=-1)) / D ** 0.5
    share = lambda x: x.unflatten(2, (Hk, rep)).sum(3)  # noqa: E731
    return {"dq": share(dq), "dk": share(dk), "dv": dv, "ddecay": dg, "dbeta": db, "dinitial_state": dh0,
            "sum_size": sum_size, "state_size": state_size, "beta_size": beta_size}


def close_grads(r, want, what="", grow=1.0):
    """dq, dk, dv, dinitial_state as outputs above.  dbeta: a dot product of 128 values that are each off by FP32_REL_L2 of
    their size.  ddecay: such dot products added over the up to 64 later tokens of a chunk (independent errors: 8 times one's),
    and <S, dS> at its end."""
    for n in ("dq", "dk", "dv"):
        close_bf16(r[n], want[n], (what, n), grow)
    if "dinitial_state" in r:
        close_fp32(r["dinitial_state"], want["dinitial_state"], (what, "dinitial_state"), grow * FP32_REL_L2, grow * FP32_MAX)
    if not want["dbeta"].numel():
        return
    biggest = lambda x: x.amax(1, keepdim=True).expand_as(x)  # noqa: E731
    tol = {"dbeta": want["beta_size"].square().mean(1, keepdim=True).sqrt() + want["beta_size"],
           "ddecay": 8 * biggest(want["sum_size"]) + biggest(want["state_size"])}
    for n, size in tol.items():
        got = r[n].double()
        assert got.shape == want[n].shape and torch.isfinite(got).all(), (what, n)
        if not got.numel():
            continue
        err, size = (got - want[n]).abs(), grow * FP32_REL_L2 * size
        bad = err > 4 * size + 2.0 ** -23 * want[n].abs()
        assert not bad.any(), (what, n, int(bad.sum()), float(err.max()), float((err / size).max()))
        assert float(err.norm()) <= float(size.norm()) + 2.0 ** -24 * float(want[n].norm()), (what, n, float(err.norm()), float(size.norm()))


def inputs(B, T, Hk, H, seed, strided=False, keys="normal", lo=1e-3, device="cuda"):
    """q, k of norm 1, v, decays spread over their logarithm between lo and 1, betas in (0, 1), and a generator."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k, v = unit(n(B, T, Hk, D)), unit(n(B, T, Hk, D)), n(B, T, H, D)
    if keys == "same":        # every key nearly the same: a triangular system far from diagonal
        k = unit(unit(n(B, 1, Hk, D)) + 0.02 * n(B, T, Hk, D))
    q, k, v = q.bfloat16(), k.bfloat16(), v.bfloat16()
    if strided:
        qkv = torch.cat([n(B, T, 8).bfloat16(), q.flatten(2), k.flatten(2), v.flatten(2), n(B, T, 8).bfloat16()], -1)
        q, k, v = (x.unflatten(2, (-1, D)) for x in qkv[..., 8:-8].split([Hk * D, Hk * D, H * D], dim=-1))
    u = torch.rand((B, T, H), generator=g, device=device)
    decay = -(lo ** u)
    beta = torch.rand((B, T, H), generator=g, device=device)
    return q, k, v, decay, beta, n


def close_bf16(got, want, what, grow=1.0):
    """Half a step of the value (2^-8 relative to it), and where terms cancel 2^-16 of the rms for the fp32 sums (some 2^8
    roundings of 2^-24 at the worst), times grow; 2^-8 in the norm."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape, what
    if not want.numel():
        return
    assert torch.isfinite(got).all(), what
    rms = want.square().mean().sqrt()
    err = (got - want).abs()
    bad = err > BF16_STEP * want.abs() + grow * 2.0 ** -16 * rms
    assert not bad.any(), (what, float(err.max()), float(rms), int(bad.sum()))
    assert float(err.norm()) <= BF16_STEP * float(want.norm()), what


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


def close_state(got, want, what, grow=1.0):
    if got.dtype is torch.bfloat16:
        close_bf16(got, want, what, grow)
    else:
        close_fp32(got, want, what, grow * FP32_REL_L2, grow * FP32_MAX)
