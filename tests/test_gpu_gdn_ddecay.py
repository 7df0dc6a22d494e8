"""ddecay of kda_gdn_bwd, token by token, for heads that remember and heads that forget: each value within what the terms that cross
its token allow (gdn_bounds), which shrinks with e^{decay}."""
import pytest
import torch

from gated_delta_rule_86_amd import gdn

from gdn_bounds import crossing_size, ddecay_is_close
from gdn_testutil import D, close_grads, gdn_ref_bwd, inputs

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


def check(args, h0=None, dht=None, cu=None, what="", grow=1.0):
    q, k, v, decay, beta, n = args
    dout = n(*v.shape).bfloat16()
    want = gdn_ref_bwd(q, k, v, decay, beta, SCALE, dout, h0, dht, cu)
    size = crossing_size(q, k, v, decay, beta, SCALE, dout, h0, dht, cu)
    c = None if cu is None else torch.tensor(cu, dtype=torch.int64, device=q.device)
    r = gdn.bwd(q, k, v, decay, beta, SCALE, dout, h0, dht, c)
    torch.cuda.synchronize()
    ddecay_is_close(r["ddecay"], want["ddecay"], size, decay, what, grow)
    if float(want["dinitial_state"].abs().amax()) < 2.0 ** -102:
        # A value below 2^-102 has no three terms of 8 bits that are all normal numbers (2^-126 and up), and smaller ones count as 0 in a
        # product.  What is left out is below 2^-126 in each of a token's 128 values: half of that in sum, signs as they fall.
        assert (r.pop("dinitial_state").double() - want["dinitial_state"]).abs().max() <= 64 * 2.0 ** -126
    close_grads(r, want, what, grow)
    return r["ddecay"], want["ddecay"]


@pytest.mark.parametrize("keys", ["normal", "same"])
@pytest.mark.parametrize("decay", [0.0, -1e-3, -0.1, -1.0, -4.0, -8.0, -12.0, -16.0, -20.0, -40.0, -80.0])
def test_one_decay(decay, keys):
    q, k, v, d, b, n = inputs(1, 200, 1, 2, 5, keys=keys)
    d = torch.full_like(d, decay)
    check((q, k, v, d, b, n), n(1, 2, D, D), n(1, 2, D, D))
    check((q, k, v, d, b, n))


@pytest.mark.parametrize("decay", [-110.0, -500.0, -999.0])
def test_nothing_is_left(decay):
    """Where the factor is 0 in fp32 the gradient is 0, not the rounding of larger numbers."""
    q, k, v, d, b, n = inputs(2, 130, 2, 2, 6)
    d = torch.full_like(d, decay)
    got, _ = check((q, k, v, d, b, n), n(2, 2, D, D), n(2, 2, D, D))
    assert (got == 0).all()


@pytest.mark.parametrize("T", [1, 2, 3, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 95, 97, 128, 129])
@pytest.mark.parametrize("lo", [1.0, 16.0])
def test_lengths(T, lo):
    """Another decay for each token, between -lo and -lo - 4."""
    q, k, v, d, b, n = inputs(2, T, 1, 2, T)
    d = -(lo + 4.0 * torch.rand(d.shape, device=d.device))
    check((q, k, v, d, b, n), n(2, 2, D, D), n(2, 2, D, D))
    check((q, k, v, d, b, n))


@pytest.mark.parametrize("lens", [[1], [5, 0, 64, 1, 63], [0, 0, 130], [65, 0], [200, 3, 128, 0, 1, 90], [700, 0, 1, 333], [10] * 60 + [900]],
                         ids=str)
def test_packed(lens):
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    q, k, v, d, b, n = inputs(1, cu[-1], 1, 2, len(lens), strided=True)
    d = d * 20.0
    check((q, k, v, d, b, n), n(len(lens), 2, D, D), n(len(lens), 2, D, D), cu)


@pytest.mark.parametrize("B,T,Hk,H", [(1, 1024, 1, 2), (2, 1500, 1, 1), (1, 2049, 1, 3)])
@pytest.mark.parametrize("most", [0.01, 1.0, 18.0])
def test_rows_cut_into_segments(B, T, Hk, H, most):
    q, k, v, d, b, n = inputs(B, T, Hk, H, T)
    check((q, k, v, most * d, b, n), n(B, H, D, D), n(B, H, D, D))


def test_mixed_gates():
    """Tokens that forget next to tokens that remember, gates that write nothing, keys and queries of 0."""
    q, k, v, d, b, n = inputs(2, 190, 2, 2, 11, lo=1e-6)
    d[:, ::9] = -14.0
    d[:, 40:50] = -1000.0
    d[:, 100] = float("-inf")
    d[:, 120:130] = 0.5
    d[0, 64:128] = -30.0
    b[:, 60:70] = 0.0
    k[:, 30:34] = 0.0
    q[:, 80:90] = 0.0
    got, want = check((q, k, v, d, b, n), n(2, 2, D, D), n(2, 2, D, D))
    outside = (d <= -1000.0) | (d > 0.0)
    assert (got[outside] == 0).all()


@pytest.mark.parametrize("decay", [-2.0, -8.0])
def test_differences(decay):
    """Central differences of <dht, final state> through the forward kernel, in the decays of one token at a time near the end."""
    q, k, v, d, b, n = inputs(1, 40, 1, 2, 23)
    d = torch.full_like(d, decay)
    h0, dht = n(1, 2, D, D), n(1, 2, D, D)
    dg = gdn.bwd(q, k, v, d, b, SCALE, torch.zeros_like(v), h0, dht)["ddecay"].double()

    def final(d):
        ht = torch.empty_like(h0)
        gdn.fwd(q, k, v, d, b, SCALE, torch.empty_like(v), h0, ht)
        return ht.double()
    e = 2.0 ** -4
    for t in (38, 39):
        x, y = d.clone(), d.clone()
        x[:, t] += e
        y[:, t] -= e
        delta = (final(x) - final(y)) / (2 * e)
        got = (delta * dht.double()).sum((-1, -2))[0]
        # fp32 rounding of a state of that many independent entries, and the third derivative: e^2 / 6 of a sum of exponentials
        # whose shares decay at least as fast as the largest
        noise = 2.0 ** -23 * float(final(d).norm()) * float(dht.norm()) / D / e
        assert ((got - dg[0, t]).abs() <= noise + e * e * dg[0, t].abs()).all(), (t, got, dg[0, t])
