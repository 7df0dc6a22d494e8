"""The operators run together as a layer uses them: projections -> q/k norm and rotation -> linear attention; a prompt, then
decode steps on the carried state; a training step through both backward passes; KDA fed by the same norm."""
import numpy as np
import pytest
import torch

from gated_delta_rule_86_amd import kda, linattn, qkrope
from gated_delta_rule_86_amd import workloads as W
from kda_testutil import check_out, run_oracle, to_device
from lin_testutil import BF16_STEP, D, close_bf16, dev, lin_ref, lin_ref_chunked
from test_gpu_qkrope import ref as rope_ref

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


def layer_inputs(B, T, Hk, H, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    qkv = n(B, T, (2 * Hk + H) * D).bfloat16()
    q, k, v = (x.unflatten(2, (-1, D)) for x in qkv.split([Hk * D, Hk * D, H * D], -1))
    decay = -torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
    f, m = qkrope.inv_freq(D, scaling="yarn", factor=4.0, original_context=4096, device="cuda")
    return q, k, v, decay, f, m, 1 + 0.1 * n(D), 1 + 0.1 * n(D), n


@pytest.mark.parametrize("T,steps", [(1, 1), (63, 2), (200, 3), (3000, 2)])
def test_prompt_then_decode(T, steps):
    """A prompt and `steps` single tokens equal one run of T + steps tokens, from positions that start far out."""
    B, Hk, H, start = 2, 2, 4, 100000
    q, k, v, decay, f, m, wq, wk, n = layer_inputs(B, T + steps, Hk, H, T)
    kw = dict(q_weight=wq, k_weight=wk, attention_factor=m)
    pos = (start + torch.arange(T + steps, device="cuda")).repeat(B, 1)
    state = (0.5 * n(B, H, D, D)).contiguous()
    h0 = state.clone()
    outs, qs, ks = [], [], []
    for lo, hi in [(0, T)] + [(T + i, T + i + 1) for i in range(steps)]:
        a, b = torch.empty(B, hi - lo, Hk, D, dtype=torch.bfloat16, device="cuda"), torch.empty(
            B, hi - lo, Hk, D, dtype=torch.bfloat16, device="cuda")
        qkrope.fwd(q[:, lo:hi], k[:, lo:hi], pos[:, lo:hi].contiguous(), f, a, b, **kw)
        o = torch.empty(B, hi - lo, H, D, dtype=torch.bfloat16, device="cuda")
        (linattn.fwd if lo == 0 else linattn.fwd_recurrent)(a, b, v[:, lo:hi], decay, SCALE, o, state, state)
        outs.append(o)
        qs.append(a)
        ks.append(b)
    # the rotated q, k are rounded once on their own (tested there); the attention starts from those values
    ro, rs = lin_ref_chunked(torch.cat(qs, 1), torch.cat(ks, 1), v, decay, SCALE, h0)
    close_bf16(torch.cat(outs, 1), ro, "out")
    assert float((state.double() - rs).norm() / rs.norm()) <= 1e-5


def test_training_step():
    """Gradients through both backward passes against automatic differentiation of the whole layer in fp64.  The chain
    rounds q', k', their gradients and the final ones to bf16, at most 2^-8 each, and dout enters exactly: four
    roundings along a path, 4 * 2^-8 in the norm."""
    B, T, Hk, H = 2, 150, 2, 4
    q, k, v, decay, f, m, wq, wk, n = layer_inputs(B, T, Hk, H, 7)
    kw = dict(q_weight=wq, k_weight=wk, attention_factor=m)
    pos = torch.arange(T, device="cuda").repeat(B, 1)
    a, b = torch.empty(B, T, Hk, D, dtype=torch.bfloat16, device="cuda"), torch.empty(
        B, T, Hk, D, dtype=torch.bfloat16, device="cuda")
    qkrope.fwd(q, k, pos, f, a, b, **kw)
    do = n(B, T, H, D).bfloat16()
    r = linattn.bwd(a, b, v, decay, SCALE, do)
    s = qkrope.bwd(q, k, pos, f, r["dq"], r["dk"], **kw)

    leaves = [x.double().contiguous().requires_grad_() for x in (q, k, v, decay, wq, wk)]
    ql, kl, vl, dl, wql, wkl = leaves
    o, _ = lin_ref(rope_ref(ql, wql, pos, f, "rms", 1e-6, False, m), rope_ref(kl, wkl, pos, f, "rms", 1e-6, False, m),
                   vl, dl, SCALE)
    want = torch.autograd.grad((o * do.double()).sum(), leaves)
    got = (s["dq"], s["dk"], r["dv"], r["ddecay"], s["dq_weight"], s["dk_weight"])
    for x, y, name in zip(got, want, ("dq", "dk", "dv", "ddecay", "dq_weight", "dk_weight")):
        rel = float((x.double() - y).norm() / y.norm())
        assert rel <= 4 * BF16_STEP, (name, rel)


def test_kda_with_outer_norm():
    """kda.fwd with use_qk_l2norm_in_kernel=False on q, k that qkrope normalised (l2) and rotated, against the oracle on the
    same bf16 values."""
    w = W.make("outer_norm", 1, 0, 2, lengths=[70, 33], seed=77, state_dtype="fp32", flags=5)
    d = to_device(w)
    g = torch.Generator(device="cuda")
    g.manual_seed(78)
    raw = [torch.randn((1, w.T, 2, 128), generator=g, device=dev()).bfloat16() for _ in range(2)]
    f, _ = qkrope.inv_freq(64, device="cuda")
    qkrope.fwd(raw[0], raw[1], None, f, d["q"], d["k"], norm="l2")
    bits = lambda x: x.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    w.q, w.k = bits(d["q"]), bits(d["k"])
    out, fin = torch.empty_like(d["q"]), torch.empty(2, 2, 128, 128, device=dev())
    kda.fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], w.scale, out, d["A_log"], d["dt_bias"], w.lower_bound, d["h0"], fin,
            d["cu"], use_qk_l2norm_in_kernel=False)
    ro, _ = run_oracle(w)
    check_out(out.float().cpu().numpy().astype(np.float64), ro, "kda")
    norms = d["q"].float().square().sum(-1).sqrt()
    # 128 channels, each rounded by at most 2^-8 of its value: the norm by at most 2^-8
    assert ((norms - 1).abs() <= BF16_STEP).all()
