"""Values that are not finite in the decayed linear attention: where they reach does not depend on how rows are cut."""
import pytest
import torch

from gated_delta_rule_86_amd import linattn
from lin_testutil import D, close_bf16, dev, lin_ref

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5
NAN = float("nan")


def fast(T, H, seed):
    """Decays near -1: a chunk of 64 tokens comes to 2^-92, so the states pass reads the two nearest chunks only."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device=dev())  # noqa: E731
    q, k, v = (n(1, T, H, D).bfloat16() for _ in range(3))
    return q, k, v, -0.9 - 0.2 * torch.rand(1, T, H, generator=g, device=dev()), n


def forward(f, q, k, v, d, h0, cu=None):
    out = torch.full_like(v, 7.0)
    ht = torch.full((1 if cu is None else len(cu) - 1, v.shape[2], D, D), 7.0, device=dev())
    f(q, k, v, d, SCALE, out, h0, ht, None if cu is None else torch.tensor(cu, device=dev()))
    return out, ht


@pytest.mark.parametrize("f", [linattn.fwd, linattn.fwd_recurrent])
@pytest.mark.parametrize("at", [0, 5, 100, 300, 700, 1500, 2500, 2999])
def test_nan_decay_lasts(f, at):
    """From the token on to the end of the row, and in the final state; the other head is left alone."""
    T = 3000
    assert linattn.workspace_size(1, T, 2) > 65536
    q, k, v, d, n = fast(T, 2, at)
    h0 = n(1, 2, D, D)
    want, ws = forward(f, q, k, v, d, h0)
    d[0, at, 1] = NAN
    out, ht = forward(f, q, k, v, d, h0)
    ro, rs = lin_ref(q[:, :, 1:], k[:, :, 1:], v[:, :, 1:], d[:, :, 1:], SCALE, h0[:, 1:])
    assert torch.isnan(rs).all() and torch.isnan(ro[:, at:]).all()
    assert torch.isnan(out[:, at:, 1].float()).all() and torch.isnan(ht[:, 1]).all()
    before = at // 64 * 64  # a chunk's tokens before it may be NaN too
    assert torch.equal(out[:, :before, 1], want[:, :before, 1])
    assert torch.equal(out[:, :, 0], want[:, :, 0]) and torch.equal(ht[:, 0], ws[:, 0])


@pytest.mark.parametrize("at", [3, 600, 1299, 1300, 2000])
def test_nan_decay_stays_in_its_sequence(at):
    q, k, v, d, n = fast(3000, 1, at)
    cu = [0, 1300, 1301, 3000]
    want, ws = forward(linattn.fwd, q, k, v, d, None, cu)
    d[0, at] = NAN
    out, ht = forward(linattn.fwd, q, k, v, d, None, cu)
    for i in range(3):
        a, b = cu[i], cu[i + 1]
        if a <= at < b:
            assert torch.isnan(out[:, at:b].float()).all() and torch.isnan(ht[i]).all()
        else:
            assert torch.equal(out[:, a:b], want[:, a:b]) and torch.equal(ht[i], ws[i])


@pytest.mark.parametrize("need_ddecay", [False, True])
@pytest.mark.parametrize("at", [70, 1500, 2990])
def test_nan_decay_in_the_backward_pass(at, need_ddecay):
    """dq from the token on; dk and dv of the tokens before it, whose share of later rows passes it, and the initial state's."""
    q, k, v, d, n = fast(3000, 1, at)
    h0, dht, do = n(1, 1, D, D), n(1, 1, D, D), n(1, 3000, 1, D).bfloat16()
    d[0, at] = NAN
    r = linattn.bwd(q, k, v, d, SCALE, do, h0, dht, need_ddecay=need_ddecay)
    assert torch.isnan(r["dq"][:, at:].float()).all()
    assert torch.isnan(r["dk"][:, :at].float()).all() and torch.isnan(r["dv"][:, :at].float()).all()
    assert torch.isnan(r["dinitial_state"]).all()
    behind = (at // 64 + 1) * 64
    assert all(torch.isfinite(r[m][:, behind:].float()).all() for m in ("dk", "dv"))
    assert torch.isfinite(r["dq"][:, :at // 64 * 64].float()).all()
    if need_ddecay:
        assert torch.isnan(r["ddecay"][:, :at]).all() and torch.isnan(r["ddecay"][:, at + 1:]).all()


@pytest.mark.parametrize("f", [linattn.fwd, linattn.fwd_recurrent])
@pytest.mark.parametrize("value", [NAN, float("inf")])
def test_initial_state_that_is_not_finite_lasts(f, value):
    """Also when its factor has long since come to 0: 0 times it is NaN."""
    q, k, v, d, n = fast(3000, 1, 1)
    h0 = n(1, 1, D, D)
    h0[0, 0, 17, 3] = value
    out, ht = forward(f, q, k, v, d, h0)
    assert not torch.isfinite(out[0, :, 0, 17].float()).any() and not torch.isfinite(ht[0, 0, 17, 3])
    other = torch.arange(D, device=dev()) != 17
    assert torch.isfinite(out[0, :, 0, other].float()).all()


@pytest.mark.parametrize("at", [10, 1400])
def test_value_that_is_not_finite(at):
    """NaN in v: its own channel of its own sequence from its chunk on; behind fast decays it lasts or is forgotten, but
    what is finite is right."""
    q, k, v, d, n = fast(3000, 1, 2)
    clean = v.clone()
    v[0, at, 0, 9] = NAN
    out, ht = forward(linattn.fwd, q, k, v, d, None)
    ro, rs = lin_ref(q, k, clean, d, SCALE)
    other = torch.arange(D, device=dev()) != 9
    close_bf16(out[..., other], ro[..., other], "out")
    assert torch.isnan(out[0, at:at + 64, 0, 9].float()).all()
    mine = out[0, :, 0, 9].float()
    close_bf16(torch.where(torch.isnan(mine), ro[0, :, 0, 9].float(), mine), ro[0, :, 0, 9], "out")
    assert torch.isfinite(mine[:at // 64 * 64]).all()


@pytest.mark.parametrize("f", [linattn.fwd, linattn.fwd_recurrent])
def test_smallest_factor(f):
    """Factors are right down to 2^-126 (e^-87.33) and 0 below it.  The exponent is rounded to fp32, 126 * 2^-24 ln 2 = 2^-17.5 of the
    factor, and the exponential by 2^-23."""
    z, big = torch.zeros(1, 1, 1, D, dtype=torch.bfloat16, device=dev()), 2.0 ** 100
    for g, normal in ((-1.0, True), (-87.0, True), (-87.33, True), (-87.34, False), (-95.0, False), (-1000.0, False)):
        d = torch.tensor([g], device=dev())
        h0, ht = torch.full((1, 1, D, D), big, device=dev()), torch.empty(1, 1, D, D, device=dev())
        f(z, z, z, d, SCALE, torch.empty_like(z), h0, ht)
        want = big * d.double().exp() if normal else torch.zeros(1, dtype=torch.float64, device=dev())
        assert ((ht.double() - want).abs() <= 2.0 ** -17 * want).all(), (g, float(ht[0, 0, 0, 0]))
