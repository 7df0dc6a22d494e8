"""Accuracy of the decayed linear attention where terms cancel: products carry 24 bits of every factor, whatever types the
states have, so what is left of terms that nearly cancel is right to fp32's roundings.  Factors cut to 16 bits fail here."""
import pytest
import torch

from gated_delta_rule_86_amd import linattn
from lin_testutil import D, dev, lin_ref, lin_ref_chunked

SCALE = D ** -0.5
gpu = pytest.mark.gpu

# The pairs below leave 2^-15 of their terms.  Per term, fp32 rounds two exponentials' arguments and results, a product with
# the scale and a row's running sum: six roundings of at most 2^-24, together 2^-22.7 at random, 2^-7.7 of what is left; out is
# rounded by 2^-9.8 (rms of half a bf16 step).  2^-6 is three times their sum.  A cut to 16 bits leaves up to 2^-18 of a term, 2^-19.3
# in the rms: 2^-4.3 of what is left (test_tolerance_tells_16_bit_factors).
PAIR_STEP = 2.0 ** -15
PAIR_TOL = 2.0 ** -6


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


def pairs(T, H, seed, device):
    """Keys, values and queries in [1, T, H, 128] and decays.  Tokens 2 j and 2 j + 1 are `twice` (equal) or `against` (opposite),
    and the decay between them is 2^-15, so each pair's share of a sum nearly cancels.  Decays stay so small that the
    roundings of their sums do not count."""
    g = torch.Generator().manual_seed(seed)
    n = lambda: (torch.randint(0, 2, (1, T // 2, H, D), generator=g) * 2 - 1).float()  # noqa: E731
    twice = lambda: n().repeat_interleave(2, 1).bfloat16().to(device)  # noqa: E731
    x = torch.randn((1, T // 2, H, D), generator=g).bfloat16()
    against = torch.stack((x, -x), 2).flatten(1, 2).to(device)
    free = n().repeat_interleave(2, 1).bfloat16().to(device)
    d = -(0.001 + 0.009 * torch.rand((1, T, H), generator=g))
    d[:, 1::2] = -PAIR_STEP
    return twice(), against, free, d.to(device)


def ref_grad(q, k, v, d, do, T):
    leaf = [x.double().requires_grad_() for x in (q, k, v)]
    o, _ = (lin_ref if T <= 64 else lin_ref_chunked)(*leaf, d, SCALE)
    return torch.autograd.grad((o * do.double()).sum(), leaf)


@gpu
@pytest.mark.parametrize("T,H", [(64, 2), (200, 2), (1400, 1)])
@pytest.mark.parametrize("state", [None, torch.bfloat16, torch.float32], ids=str)
def test_weights_and_rows(T, H, state):
    """Sources in pairs that cancel: the weights within a chunk, the weighted rows on their way into the state, and a cut row."""
    k, v, q, d = pairs(T, H, 5 + T, dev())
    ht = None if state is None else torch.empty(1, H, D, D, dtype=state, device=dev())
    want, ws = lin_ref_chunked(q, k, v, d, SCALE)
    odd = slice(1, None, 2)  # even tokens see half a pair
    for f in (linattn.fwd, linattn.fwd_recurrent):
        out = torch.empty_like(v)
        f(q, k, v, d, SCALE, out, None, ht)
        assert rel(out[:, odd], want[:, odd]) <= PAIR_TOL, f.__name__
        if ht is not None:
            assert rel(ht, ws) <= PAIR_TOL, f.__name__


@gpu
@pytest.mark.parametrize("T,Hk,H", [(64, 2, 2), (200, 2, 2), (1400, 1, 2)])
@pytest.mark.parametrize("need_ddecay", [False, True])
def test_gradients(T, Hk, H, need_ddecay):
    """The same for dq (keys against), dk (gradients of out against) and dv (queries against); shared heads too."""
    twice, against, free, d = pairs(T, H, 9 + T, dev())
    few = lambda x: x[:, :, :Hk].contiguous()  # noqa: E731
    odd, even = slice(1, None, 2), slice(0, None, 2)
    for name, (q, k, v, do), at in (("dq", (free, against, twice, free), odd), ("dk", (twice, free, free, against), even),
                                    ("dv", (against, free, free, twice), even)):
        q, k = few(q), few(k)
        r = linattn.bwd(q, k, v, d, SCALE, do, need_ddecay=need_ddecay)
        want = dict(zip(("dq", "dk", "dv"), ref_grad(q, k, v, d, do, T)))
        assert rel(r[name][:, at], want[name][:, at]) <= PAIR_TOL, name


@gpu
@pytest.mark.parametrize("T", [64, 1984])
@pytest.mark.parametrize("h0_dt,ht_dt", [(None, None), (None, torch.bfloat16), (None, torch.float32),
                                         (torch.bfloat16, None), (torch.bfloat16, torch.bfloat16),
                                         (torch.float32, torch.float32)], ids=str)
def test_state_share(T, h0_dt, ht_dt):
    """A state whose entries are h + m + r, with bits in the places of three bf16 terms, next to -(h + m): the queries of the last
    chunk see the sum of the r alone, 64 r = 2^-13 scale.  fp32 leaves 24 products' sums of 2^-24 to 2^-22 each, 2^-4 of it
    at most; two terms would leave 0.  At T = 1984 the state crosses segments."""
    assert (linattn.workspace_size(1, T + 64, 1) > 65536) == (T > 1000)
    g = torch.Generator().manual_seed(3)
    h = 1.0 + torch.randint(0, 128, (D,), generator=g) / 128.0
    m = (1.0 + torch.randint(0, 128, (D,), generator=g) / 128.0) * 2.0 ** -10
    r = torch.full((D,), 2.0 ** -19)
    sign = torch.tensor([1.0, -1.0]).repeat(D // 2)
    q, k, v = (torch.zeros(1, T + 64, 1, D) for _ in range(3))
    v[0, 0, 0], v[0, 1, 0], v[0, 2, 0] = h, m, r
    k[0, 0, 0] = k[0, 1, 0] = sign
    k[0, 2, 0, ::2] = 1.0
    q[0, T:] = 1.0
    q, k, v = (x.bfloat16().to(dev()) for x in (q, k, v))
    d = torch.zeros(1, device=dev())
    state = lambda t: None if t is None else torch.zeros(1, 1, D, D, dtype=t, device=dev())  # noqa: E731
    want = torch.full((D,), 64 * 2.0 ** -19 * SCALE, dtype=torch.float64, device=dev())
    for f in (linattn.fwd, linattn.fwd_recurrent):
        out = torch.empty_like(v)
        f(q, k, v, d, SCALE, out, state(h0_dt), state(ht_dt))
        err = (out[0, T:, 0].double() - want).abs()
        assert float(err.max()) <= 2.0 ** -3 * float(want[0]), (f.__name__, float(err.max()))


@gpu
@pytest.mark.parametrize("T,H", [(130, 2), (3000, 1)])
def test_out_does_not_depend_on_the_final_state(T, H):
    g = torch.Generator(device=dev()).manual_seed(1)
    q, k, v = (torch.randn(1, T, H, D, generator=g, device=dev()).bfloat16() for _ in range(3))
    d = -0.05 * torch.rand(1, T, H, generator=g, device=dev())
    got = []
    for dt in (None, torch.bfloat16, torch.float32):
        ht = None if dt is None else torch.empty(1, H, D, D, dtype=dt, device=dev())
        got.append(torch.empty_like(v))
        linattn.fwd(q, k, v, d, SCALE, got[-1], None, ht)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_tolerance_tells_16_bit_factors():
    """The oracle in fp32, with its weights cut to two bf16 terms: off by more than the tolerance; uncut: within."""
    T = 64
    k, v, q, d = pairs(T, 2, 5, "cpu")
    want, _ = lin_ref(q, k, v, d, SCALE)
    c = d.double().cumsum(1)
    low = torch.ones(T, T, dtype=torch.bool).tril()
    w = torch.einsum("bthd,bshd->bhts", q.float(), k.float()) * SCALE
    w = (w * (c[:, :, None] - c[:, None]).permute(0, 3, 1, 2).exp().float()).masked_fill(~low, 0.0)
    for cut, most in ((False, PAIR_TOL), (True, None)):
        p = w
        if cut:
            hi = w.bfloat16().float()
            p = hi + (w - hi).bfloat16().float()
        out = torch.einsum("bhts,bshd->bthd", p.double(), v.double()).float().bfloat16()
        off = rel(out[:, 1::2], want[:, 1::2])
        assert off <= most if most else off > 2 * PAIR_TOL, off
