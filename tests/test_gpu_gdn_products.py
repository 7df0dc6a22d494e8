"""Products of two fp32 factors in the gated delta rule: what their 16-bit terms leave out has no sign.

Two tokens write to a state whose columns 0 and 1 are s and -s, with v = 0, no decay, k_0 = e_0 and k_1 = e_0 + e_1.  The first
token's residual is -s; the second reads s - s = 0 and gets, through the triangular system, beta_0 s: one product of two factors
of 24 bits.  Column 1 becomes -s + beta_0 s.

What may be off, with e = 2^-24, relative to |s|: the product's sum and the three steps that add the terms of a write to the state round
to the nearest at full size, by at most e each with either sign (steps before them are 2^-7 and less in size); what a product
leaves out is at most 2^-22.4.  One value: 4 e + 2^-22.4 < 2^-21.  The roundings are evenly spread within half a step, e / sqrt(3) root
mean square at the most, sqrt(4 / 3) e together with their signs independent, and what is left out 2^-25.7: below 1.3 e.  The mean
over n independent samples is then within six times 1.3 e / sqrt(n).  Terms cut towards zero in both factors leave out mid lo + lo
mid + lo lo always on the same side: 2^-25 of |s| in the mean, ten times that."""
import pytest
import torch

from gated_delta_rule_86_amd import gdn

from gdn_testutil import D

pytestmark = pytest.mark.gpu


def problem(H, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = 1.0 + torch.rand((1, H, D), generator=g, device="cuda")
    s = torch.where(torch.rand(s.shape, generator=g, device="cuda") < 0.5, -s, s)
    beta = 0.5 + 0.5 * torch.rand((1, 2, H), generator=g, device="cuda")
    beta[:, 1] = 1.0
    k = torch.zeros(1, 2, 1, D, dtype=torch.bfloat16, device="cuda")
    k[0, 0, 0, 0] = k[0, 1, 0, 0] = k[0, 1, 0, 1] = 1.0
    h0 = torch.zeros(1, H, D, D, device="cuda")
    h0[..., 0], h0[..., 1] = s, -s
    return s, beta, k, h0


def test_products_have_no_side():
    H = 256
    s, beta, k, h0 = problem(H, 1)
    v = torch.zeros(1, 2, H, D, dtype=torch.bfloat16, device="cuda")
    ht = torch.empty_like(h0)
    gdn.fwd(torch.zeros_like(k), k, v, torch.zeros_like(beta), beta, 1.0, torch.empty_like(v), h0, ht)
    b, x = beta[:, 0, :, None].double(), s.double()
    err = (ht[..., 1].double() - (b * x - x)) / x
    print(f"forward: mean {float(err.mean()):.3e} rms {float(err.square().mean().sqrt()):.3e} of 2^-24 = {2.0 ** -24:.3e}")
    assert err.abs().max() <= 2.0 ** -21
    assert err.mean().abs() <= 6 * 1.3 * 2.0 ** -24 / (H * D) ** 0.5


def test_products_of_the_backward_pass_have_no_side():
    """The same with time turned: the state's gradient has columns s and -s behind the tokens, k_1 = e_0 and k_0 = e_0 + e_1.  dw_1 = s; token
    0 reads s - s = 0 and gets -beta_1 s; dL/dS before them is dL/dS - dx_0 k_0 - dx_1 k_1, column 1: -s + beta_1 s with beta_0 = 1."""
    H = 256
    s, beta, k, dht = problem(H, 2)
    beta, k = beta.flip(1).contiguous(), k.flip(1).contiguous()
    v = torch.zeros(1, 2, H, D, dtype=torch.bfloat16, device="cuda")
    r = gdn.bwd(torch.zeros_like(k), k, v, torch.zeros_like(beta), beta, 1.0, v, None, dht)
    b, x = beta[:, 1, :, None].double(), s.double()
    err = (r["dinitial_state"][..., 1].double() - (b * x - x)) / x
    print(f"backward: mean {float(err.mean()):.3e} rms {float(err.square().mean().sqrt()):.3e} of 2^-24 = {2.0 ** -24:.3e}")
    assert err.abs().max() <= 2.0 ** -21
    assert err.mean().abs() <= 6 * 1.3 * 2.0 ** -24 / (H * D) ** 0.5
