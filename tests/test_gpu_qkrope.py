"""q/k norm with position rotation (kda_qk_rope, kda_qk_rope_bwd) against plain 64-bit references.

Tolerances: an output is rounded once from fp32 (half a step, eps / 2 of its value).  Before that each value sees
under ten fp32 roundings (square sum of D <= 512 channels in a tree of at most 16 + 5 steps under the root, factor,
weight, rotation with a cancelling difference, sin and cos to 2^-23): 16 * 2^-24 of the size of its pair.  Weight
gradients sum B T heads terms: each is off by at most 2^-20 of its own size, independently, so the norm of their
errors stays below 2^-20 sqrt(count) rms; the running sums add 2^-24 per step to partial sums of that size.
"""
import math

import pytest
import torch

from gated_delta_rule_86_amd import qkrope

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def ref(x, w, pos, f, norm, eps, inter, m):
    """fp64, differentiable."""
    D = x.shape[-1]
    R = 0 if f is None else 2 * f.numel()
    ss = (x * x).sum(-1, keepdim=True)
    n = x
    if norm == "rms":
        n = x / (ss / D + eps).sqrt()
    elif norm == "l2":
        n = x / (ss + eps).sqrt()
    if w is not None:
        n = n * w
    if R == 0:
        return n
    t = (pos.double()[..., None] * f.double())[:, :, None]
    c, s = m * t.cos(), m * t.sin()
    h = n[..., :R]
    a, b = (h[..., 0::2], h[..., 1::2]) if inter else (h[..., :R // 2], h[..., R // 2:])
    u, v = a * c - b * s, a * s + b * c
    h = torch.stack((u, v), -1).flatten(-2) if inter else torch.cat((u, v), -1)
    return torch.cat((h, n[..., R:]), -1)


def make(B, T, Hq, Hk, D, R, dtype, seed, fused=False, far=1 << 20, weights=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if fused:
        x = n(B, T, (Hq + Hk) * D + 16).to(dtype)[..., 8:-8]
        q, k = (y.unflatten(2, (-1, D)) for y in x.split([Hq * D, Hk * D], -1))
    else:
        q, k = n(B, T, Hq, D).to(dtype), n(B, T, Hk, D).to(dtype)
    pos = torch.randint(0, far, (B, T), generator=g, device="cuda")
    f = None if R == 0 else qkrope.inv_freq(R, device="cuda")[0]
    w = (1 + 0.2 * n(D), 1 + 0.2 * n(D)) if weights else (None, None)
    return q, k, pos, f, w, n


def check_rows(got, want, dtype, what):
    """Element by element: half a step of the value and 16 fp32 roundings of the head's rms."""
    size = want.square().mean(-1, keepdim=True).sqrt()
    tol = torch.finfo(dtype).eps / 2 * want.abs() + 16 * 2.0 ** -24 * (want.abs() + 4 * size)
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25  # half a step of its subnormal numbers
    assert got.dtype == dtype and torch.isfinite(got).all(), what
    err = (got.double() - want).abs()
    assert (err <= tol).all(), (what, float(err.max()), float((err / tol).max()))


CASES = [
    # B, T, Hq, Hk, D, R, dtype, norm, interleaved, fused, weights
    (1, 1, 1, 1, 128, 128, "bf16", "rms", False, False, True),
    (2, 3, 5, 1, 128, 128, "bf16", "rms", True, True, True),
    (1, 67, 32, 8, 128, 64, "bf16", "l2", False, True, False),
    (3, 33, 4, 2, 64, 64, "fp16", "rms", False, True, True),
    (1, 130, 3, 3, 256, 128, "fp32", "rms", True, False, True),
    (2, 65, 7, 2, 512, 512, "fp32", "l2", False, False, True),
    (1, 40, 2, 2, 16, 16, "bf16", "rms", False, False, True),
    (1, 41, 6, 3, 80, 32, "fp16", None, True, False, False),
    (2, 29, 4, 4, 48, 0, "fp32", "rms", False, True, True),
    (1, 2000, 12, 4, 128, 128, "bf16", "rms", False, True, True),
    (1, 9, 2, 1, 144, 144, "fp32", None, False, False, True),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    B, T, Hq, Hk, D, R, dt, norm, inter, fused, weights = case
    q, k, pos, f, w, n = make(B, T, Hq, Hk, D, R, DT[dt], 1 + T, fused, weights=weights)
    qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    kw = dict(q_weight=w[0], k_weight=w[1], norm=norm, interleaved=inter, attention_factor=1.25)
    qkrope.fwd(q, k, pos, f, qo, ko, **kw)
    for got, x, wt, what in ((qo, q, w[0], "q"), (ko, k, w[1], "k")):
        want = ref(x.double(), None if wt is None else wt.double(), pos, f, norm, 1e-6, inter, 1.25)
        check_rows(got, want, DT[dt], what)
    # in place, through views of one buffer: the same bits, and nothing else in the buffer moves
    q2, k2 = q.clone(), k.clone()
    if fused:
        base = torch.full((B, T, (Hq + Hk) * D + 16), 7.0, dtype=DT[dt], device="cuda")
        q2, k2 = (y.unflatten(2, (-1, D)) for y in base[..., 8:-8].split([Hq * D, Hk * D], -1))
        q2.copy_(q)
        k2.copy_(k)
    qkrope.fwd(q2, k2, pos, f, q2, k2, **kw)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    if fused:
        assert (base[..., :8] == 7).all() and (base[..., -8:] == 7).all()


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    B, T, Hq, Hk, D, R, dt, norm, inter, fused, weights = case
    q, k, pos, f, w, n = make(B, T, Hq, Hk, D, R, DT[dt], 50 + T, fused, weights=weights)
    dqo, dko = n(*q.shape).to(DT[dt]), n(*k.shape).to(DT[dt])
    kw = dict(q_weight=w[0], k_weight=w[1], norm=norm, interleaved=inter, attention_factor=0.75)
    r = qkrope.bwd(q, k, pos, f, dqo, dko, **kw)
    assert ("dq_weight" in r) == weights
    for x, dy, wt, name in ((q, dqo, w[0], "q"), (k, dko, w[1], "k")):
        xl = x.double().contiguous().requires_grad_()
        wl = None if wt is None else wt.double().requires_grad_()
        y = ref(xl, wl, pos, f, norm, 1e-6, inter, 0.75)
        g = torch.autograd.grad((y * dy.double()).sum(), [xl] if wl is None else [xl, wl])
        check_rows(r["d" + name], g[0], DT[dt], "d" + name)
        if wl is not None:
            count = x.numel() // D
            err = (r[f"d{name}_weight"].double() - g[1]).abs()
            # a term dn x r has size about 1: 2^-20 sqrt(count), four sigma, and 2^-24 per step of the sums
            tol = (4 * 2.0 ** -20 + 2.0 ** -24 * math.sqrt(count)) * math.sqrt(count) * 2
            assert (err <= tol).all(), (name, float(err.max()), tol)
    assert torch.equal(qkrope.bwd(q, k, pos, f, dqo, dko, **kw)["dq"], r["dq"])
    if weights:
        again = qkrope.bwd(q, k, pos, f, dqo, dko, **kw)
        assert torch.equal(again["dq_weight"], r["dq_weight"]) and torch.equal(again["dk_weight"], r["dk_weight"])


def test_backward_differences():
    q, k, pos, f, w, n = make(1, 6, 2, 1, 32, 16, torch.float32, 3, far=100)
    dqo, dko = n(*q.shape), n(*k.shape)
    r = qkrope.bwd(q, k, pos, f, dqo, dko, q_weight=w[0], k_weight=w[1])

    def loss(q, k, wq, wk):
        return float((ref(q, wq, pos, f, "rms", 1e-6, False, 1.0) * dqo.double()).sum()
                     + (ref(k, wk, pos, f, "rms", 1e-6, False, 1.0) * dko.double()).sum())
    args = [x.double() for x in (q, k, *w)]
    for i, name in enumerate(("dq", "dk", "dq_weight", "dk_weight")):
        u = n(*args[i].shape).double()
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + 1e-5 * u, args[i] - 1e-5 * u
        want = (loss(*hi) - loss(*lo)) / 2e-5
        got = float((r[name].double() * u).sum())
        # fp32 values, 2^-20 each; central differences of fp64: step^2 and 2^-52 / step
        assert abs(got - want) <= 2.0 ** -18 * float(r[name].double().norm() * u.norm()) + 1e-6, (name, got, want)


def test_positions():
    """None counts from 0 in each row; far and negative positions keep fp32 accuracy."""
    q, k, _, f, _, _ = make(2, 50, 2, 2, 128, 128, torch.float32, 5)
    a, b = torch.empty_like(q), torch.empty_like(k)
    c, d = torch.empty_like(q), torch.empty_like(k)
    qkrope.fwd(q, k, None, f, a, b)
    qkrope.fwd(q, k, torch.arange(50, device="cuda").repeat(2, 1), f, c, d)
    assert torch.equal(a, c) and torch.equal(b, d)
    pos = torch.tensor([[-5, -(1 << 20), (1 << 26) + 3, 1 << 24, (1 << 20) + 1] * 10] * 2, device="cuda")
    qkrope.fwd(q, k, pos, f, a, b, norm=None)
    check_rows(a, ref(q.double(), None, pos, f, None, 0, False, 1.0), torch.float32, "far")


def test_special_values():
    """A row of zeros stays zero with a finite gradient; a NaN stays in its own head; no eps and no norm."""
    q, k, pos, f, w, n = make(1, 8, 2, 1, 64, 64, torch.float32, 6)
    q[0, 3] = 0.0
    q[0, 5, 1, 7] = float("nan")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    qkrope.fwd(q, k, pos, f, qo, ko, q_weight=w[0])
    assert (qo[0, 3] == 0).all() and torch.isnan(qo[0, 5, 1]).any()
    ok = torch.ones(8, 2, dtype=torch.bool)
    ok[5, 1] = False
    assert torch.isfinite(qo[0][ok.cuda()]).all()
    r = qkrope.bwd(q, k, pos, f, torch.ones_like(q), torch.ones_like(k), q_weight=w[0])
    assert torch.isfinite(r["dq"][0, 3]).all() and torch.isfinite(r["dk"]).all()


def test_empty():
    q, k = torch.empty(2, 0, 3, 64, device="cuda"), torch.empty(2, 0, 1, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    f, _ = qkrope.inv_freq(64, device="cuda")
    qkrope.fwd(q, k, None, f, q.clone(), k.clone())
    r = qkrope.bwd(q, k, None, f, q.clone(), k.clone(), q_weight=w, k_weight=w)
    assert r["dq"].shape == q.shape and (r["dq_weight"] == 0).all() and (r["dk_weight"] == 0).all()


def test_stream_and_graph():
    q, k, pos, f, w, n = make(1, 300, 4, 2, 128, 128, torch.bfloat16, 8)
    qo, ko, dqo, dko = torch.empty_like(q), torch.empty_like(k), n(*q.shape).bfloat16(), n(*k.shape).bfloat16()
    kw = dict(q_weight=w[0], k_weight=w[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        qkrope.fwd(q, k, pos, f, qo, ko, **kw)
        qkrope.bwd(q, k, pos, f, dqo, dko, **kw)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qkrope.fwd(q, k, pos, f, qo, ko, **kw)
        r = qkrope.bwd(q, k, pos, f, dqo, dko, **kw)
    for _ in range(3):
        q.copy_(n(*q.shape).bfloat16())
        pos.add_(1000)
        a, b = torch.empty_like(q), torch.empty_like(k)
        qkrope.fwd(q, k, pos, f, a, b, **kw)
        e = qkrope.bwd(q, k, pos, f, dqo, dko, **kw)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, a) and torch.equal(ko, b)
        assert all(torch.equal(r[m], e[m]) for m in ("dq", "dk", "dq_weight", "dk_weight"))
    side.wait_stream(torch.cuda.current_stream())
    qkrope.fwd(q, k, pos, f, qo.zero_(), ko, **kw, stream=side)
    side.synchronize()
    assert torch.equal(ko, b)


def test_strides_past_32_bits():
    """Batch rows 2^31 elements apart, in place, equal their copies."""
    T, D, R = 37, 128, 64
    base = torch.empty((1 << 31) + T * 4 * D, dtype=torch.bfloat16, device="cuda")
    q, k, pos, f, w, n = make(2, T, 3, 1, D, R, torch.bfloat16, 9)
    x = base.as_strided((2, T, 4, D), (1 << 31, 4 * D, D, 1))
    x[:, :, :3].copy_(q)
    x[:, :, 3:].copy_(k)
    a, b = torch.empty(2, T, 3, D, dtype=torch.bfloat16, device="cuda"), torch.empty(2, T, 1, D, dtype=torch.bfloat16,
                                                                                     device="cuda")
    kw = dict(q_weight=w[0], k_weight=w[1])
    qc, kc = x[:, :, :3].contiguous(), x[:, :, 3:].contiguous()
    qkrope.fwd(qc, kc, pos, f, a, b, **kw)
    r = qkrope.bwd(qc, kc, pos, f, a, b, **kw)
    e = qkrope.bwd(x[:, :, :3], x[:, :, 3:], pos, f, a, b, **kw)
    assert all(torch.equal(r[m], e[m]) for m in r)
    qkrope.fwd(x[:, :, :3], x[:, :, 3:], pos, f, x[:, :, :3], x[:, :, 3:], **kw)
    assert torch.equal(x[:, :, :3], a) and torch.equal(x[:, :, 3:], b)
