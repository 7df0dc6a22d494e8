"""The bounds of the decays' gradients (gdn_bounds): what they accept and what they reject, and the reference's gradient of heads that
forget fast (no GPU)."""
import pytest
import torch

from gdn_bounds import crossing_size, ddecay_is_close
from gdn_testutil import D, FP32_REL_L2, gdn_ref, gdn_ref_bwd, inputs

SCALE = D ** -0.5


def problem(decay, keys="normal", T=70):
    q, k, v, d, b, n = inputs(1, T, 1, 2, 3, keys=keys, device="cpu")
    d = torch.full_like(d, decay)
    h0, dht, dout = n(1, 2, D, D), n(1, 2, D, D), n(*v.shape).bfloat16()
    want = gdn_ref_bwd(q, k, v, d, b, SCALE, dout, h0, dht)
    return want, crossing_size(q, k, v, d, b, SCALE, dout, h0, dht), d, (q, k, v, b, n, h0, dht, dout)


@pytest.mark.parametrize("keys", ["normal", "same"])
@pytest.mark.parametrize("decay", [-0.01, -1.0, -8.0, -12.0, -16.0, -20.0, -60.0])
def test_what_is_accepted_and_rejected(decay, keys):
    want, size, d, _ = problem(decay, keys)
    dg = want["ddecay"]
    ddecay_is_close(dg.float(), dg, size, d)
    with pytest.raises(AssertionError):
        ddecay_is_close(torch.zeros_like(dg), dg, size, d)
    with pytest.raises(AssertionError):
        ddecay_is_close(dg * (1 + 1e-2), dg, size, d)
    if decay <= -8.0:   # one rounding of the token's own read and write
        noise = 2.0 ** -24 * want["sum_size"] * torch.randn(dg.shape, generator=torch.Generator().manual_seed(1))
        with pytest.raises(AssertionError):
            ddecay_is_close(dg + noise, dg, size, d)


def test_a_decay_that_leaves_nothing():
    want, size, d, _ = problem(-120.0)
    ddecay_is_close(torch.zeros_like(want["ddecay"]), want["ddecay"], size, d)
    with pytest.raises(AssertionError):
        ddecay_is_close(torch.full_like(want["ddecay"], 1e-7), want["ddecay"], size, d)


def test_size_bounds_the_gradient():
    for decay in (-0.01, -3.0, -16.0):
        want, (size, _), _, _ = problem(decay)
        assert (want["ddecay"].abs() <= 2 * size).all() and (size * FP32_REL_L2 / D ** 0.5 < 1e-2 * want["ddecay"].abs().max()).all()


@pytest.mark.parametrize("decay", [-8.0, -16.0, -40.0])
def test_reference_of_heads_that_forget(decay):
    """The recurrence run backwards keeps its digits where the gradient is e^{g}-sized: against automatic differentiation, and that
    against differences of the loss in one token's decay at a time."""
    want, _, d, (q, k, v, b, n, h0, dht, dout) = problem(decay, T=6)
    leaf = d.double().requires_grad_()

    def loss(d):
        out, fin = gdn_ref(q, k, v, d, b, SCALE, h0)
        return (out * dout.double()).sum() + (fin * dht.double()).sum()
    grad, = torch.autograd.grad(loss(leaf), leaf)
    assert (want["ddecay"] - grad).abs().max() <= 1e-10 * grad.abs().max()
    if decay == -8.0:
        with torch.no_grad():
            for t in range(6):
                e = torch.zeros_like(leaf)
                e[0, t, 1] = 1e-3
                got = (loss(leaf + e) - loss(leaf - e)) / 2e-3
                assert abs(got - grad[0, t, 1]) <= 1e-5 * grad.abs().max()
