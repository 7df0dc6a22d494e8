"""kda_gdn_bwd against the recurrence run backwards in 64 bits, on the GPU."""
import pytest
import torch

from gated_delta_rule_86_amd import gdn

from gdn_testutil import D, close_grads, gdn_ref, gdn_ref_bwd, inputs

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


def check(args, h0=None, dht=None, cu=None, what="", grow=1.0, **kw):
    q, k, v, decay, beta, n = args
    dout = n(*v.shape).bfloat16()
    want = gdn_ref_bwd(q, k, v, decay, beta, SCALE, dout, h0, dht, cu)
    c = None if cu is None else torch.tensor(cu, dtype=torch.int64, device=q.device)
    r = gdn.bwd(q, k, v, decay, beta, SCALE, dout, h0, dht, c, **kw)
    torch.cuda.synchronize()
    close_grads(r, want, what, grow)
    return r


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200])
def test_lengths(T):
    args = inputs(2, T, 2, 2, T)
    n = args[-1]
    check(args, n(2, 2, D, D), n(2, 2, D, D))
    check(args)


@pytest.mark.parametrize("Hk,H", [(1, 1), (1, 3), (2, 4), (3, 3), (2, 8)])
@pytest.mark.parametrize("strided", [False, True])
def test_heads_and_strides(Hk, H, strided):
    args = inputs(2, 97, Hk, H, 7 * H + Hk, strided=strided)
    n = args[-1]
    check(args, n(2, H, D, D), n(2, H, D, D))


@pytest.mark.parametrize("h0", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dht", [False, True])
@pytest.mark.parametrize("need", [False, True])
def test_states(h0, dht, need):
    args = inputs(3, 70, 2, 2, 5)
    n = args[-1]
    r = check(args, None if h0 is None else n(3, 2, D, D).to(h0), n(3, 2, D, D) if dht else None, need_dinitial_state=need)
    assert ("dinitial_state" in r) == need


@pytest.mark.parametrize("lens", [[1], [5, 0, 64, 1, 63], [0, 0, 130], [64, 64], [65, 0], [0], [200, 3, 128, 0, 1, 90]], ids=str)
def test_packed(lens):
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    args = inputs(1, cu[-1], 1, 2, len(lens))
    n = args[-1]
    check(args, n(len(lens), 2, D, D), n(len(lens), 2, D, D), cu)


@pytest.mark.parametrize("B,T,Hk,H", [(1, 1024, 1, 2), (2, 1500, 1, 1), (1, 2049, 3, 3)])
def test_rows_cut_into_segments(B, T, Hk, H):
    args = inputs(B, T, Hk, H, T, lo=1e-4)
    n = args[-1]
    check(args, n(B, H, D, D), n(B, H, D, D))
    check(args)


@pytest.mark.parametrize("lens", [[700, 0, 1, 333], [1500], [10] * 60 + [900], [256, 256, 256, 256], [257, 255, 600],
                                  [0, 640, 0, 640, 0], [63, 1, 1000, 2]], ids=str)
def test_packed_and_cut(lens):
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    args = inputs(1, cu[-1], 1, 2, len(lens), lo=1e-4)
    n = args[-1]
    check(args, n(len(lens), 2, D, D), n(len(lens), 2, D, D), cu)


@pytest.mark.parametrize("keys", ["normal", "same"])
@pytest.mark.parametrize("beta", [0.0, 1.0, 2.0])
@pytest.mark.parametrize("decay", [0.0, -0.01, -20.0, -1000.0, float("-inf")])
def test_gates(keys, beta, decay):
    q, k, v, d, b, n = inputs(1, 150, 1, 2, 3, keys=keys)
    d = torch.full_like(d, decay)
    b = torch.full_like(b, beta)
    if decay == -1000.0:
        d[:, ::7] = 0.0
    # beta 2 and one key for all tokens: nothing damps an error of the states or of their gradients, see the forward test
    check((q, k, v, d, b, n), n(1, 2, D, D), n(1, 2, D, D), grow=12.0 if beta == 2.0 else 1.0)


def test_mixed_gates():
    q, k, v, d, b, n = inputs(2, 190, 2, 2, 11, lo=1e-6)
    d[:, 40:50] = -1000.0
    d[:, 100] = float("-inf")
    d[:, 120:130] = 0.5
    d[0, 64:128] = -30.0
    b[:, 60:70] = 0.0
    k[:, 30:34] = 0.0
    q[:, 80:90] = 0.0
    check((q, k, v, d, b, n), n(2, 2, D, D), n(2, 2, D, D))


def test_differences():
    """Central differences of a loss through the forward kernel's own outputs, along random directions of the fp32 inputs (the
    gates and the initial state), with the state alone as output: bf16 rounding of out stays out of it."""
    q, k, v, d, b, n = inputs(1, 130, 1, 2, 23)
    d = d.clamp(max=-0.01)
    h0, dht = n(1, 2, D, D), n(1, 2, D, D)
    r = gdn.bwd(q, k, v, d, b, SCALE, torch.zeros_like(v), h0, dht)

    def loss(d, b, h0):
        ht = torch.empty_like(h0)
        gdn.fwd(q, k, v, d, b, SCALE, torch.empty_like(v), h0, ht)
        return (ht.double() * dht.double()).sum()
    size = float(gdn_ref(q, k, v, d, b, SCALE, h0)[1].norm() * dht.double().norm())
    for name, x in (("ddecay", d), ("dbeta", b), ("dinitial_state", h0)):
        u = n(*x.shape)
        u *= x.norm() / u.norm()
        e = 2.0 ** -7 if name == "dinitial_state" else 2.0 ** -9
        plus, minus = ([x + s * e * u if x is y else y for y in (d, b, h0)] for s in (1, -1))
        got = (loss(*plus) - loss(*minus)) / (2 * e)
        want = (r[name].double() * u.double()).sum()
        # the state's fp32 error (5e-6 of its size at the most, spread over independent entries) against the step, and the third
        # derivative's e^2
        assert abs(got - want) <= 5e-6 * size / D / e + e * e * 40 * size / D, (name, float(got), float(want))


def test_bad_lengths():
    q, k, v, d, b, n = inputs(1, 20, 1, 2, 9)
    dht = n(3, 2, D, D)
    r = gdn.bwd(q, k, v, d, b, SCALE, torch.ones_like(v), None, dht, torch.tensor([0, 5, 4, 20], device=q.device))
    assert gdn.device_status(r["workspace"]) != 0 and torch.equal(r["dinitial_state"], dht)


def test_no_tokens():
    q, k, v, d, b, n = inputs(2, 0, 1, 2, 9)
    dht = n(2, 2, D, D)
    r = gdn.bwd(q, k, v, d, b, SCALE, torch.ones_like(v), None, dht)
    assert torch.equal(r["dinitial_state"], dht) and r["dq"].shape == q.shape


def test_repeats():
    q, k, v, d, b, n = inputs(1, 1300, 1, 2, 17)
    dout, h0 = n(*v.shape).bfloat16(), n(1, 2, D, D)
    x, y = (gdn.bwd(q, k, v, d, b, SCALE, dout, h0, h0) for _ in range(2))
    assert all(torch.equal(x[m], y[m]) for m in x if m != "workspace")


@pytest.mark.parametrize("lo,hi", [(0.05, 0.5), (1.0, 20.0), (0.0, 3.0)], ids=str)
def test_cut_rows_that_forget(lo, hi):
    q, k, v, d, b, n = inputs(1, 2000, 1, 3, 31)
    d = -(lo + (hi - lo) * torch.rand(d.shape, device=d.device))
    d[:, :, 2] *= 1e-3
    check((q, k, v, d, b, n), n(1, 3, D, D), n(1, 3, D, D))
    check((q, k, v, d, b, n), n(3, 3, D, D), n(3, 3, D, D), [0, 900, 901, 2000])


def test_gradient_that_is_not_finite_lasts():
    """A row of dfinal_state that is not finite reaches the start of its sequence, over cuts and strong decays, and no other row."""
    q, k, v, d, b, n = inputs(1, 2500, 1, 2, 33)
    d = torch.full_like(d, -5.0)
    dout, h0, dht = n(*v.shape).bfloat16(), n(1, 2, D, D), n(1, 2, D, D)
    clean = gdn.bwd(q, k, v, d, b, SCALE, dout, h0, dht)
    dht[0, 1, 7, 9] = float("nan")
    r = gdn.bwd(q, k, v, d, b, SCALE, dout, h0, dht)
    keep = torch.ones(D, dtype=torch.bool, device=q.device)
    keep[7] = False
    assert torch.equal(r["dinitial_state"][:, 1, keep], clean["dinitial_state"][:, 1, keep])
    assert torch.equal(r["dv"][:, :, 1, keep], clean["dv"][:, :, 1, keep]) and torch.equal(r["dv"][:, :, 0], clean["dv"][:, :, 0])
    assert r["dinitial_state"][0, 1, 7].isnan().all() and r["dv"][:, :, 1, 7].isnan().all()
