"""The gated delta rule over rows that are cut into segments: bf16 states, lengths that are not valid, values that are not finite."""
import pytest
import torch

from gated_delta_rule_86_amd import gdn

from gdn_testutil import D, close_grads, gdn_ref_bwd, inputs
from test_gpu_gdn import check, run

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


def is_cut(B, T, H, N=0):
    """The workspace holds the states of the cuts, three for each segment and head, behind the records."""
    records = (B * T // 32 + (N or B) + 1) * H * 13312
    return gdn.workspace_size(B, T, H, N, bool(N)) >= 256 + records + 2 * 3 * H * D * D * 4


def offsets(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


@pytest.mark.parametrize("B,T,H", [(1, 1024, 2), (2, 1500, 1), (1, 2049, 3)])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("most", [1.0, 1e-2])
def test_bf16_states(B, T, H, in_place, most):
    """Carried in place too: the segments that end a sequence write over the state that its first one still reads."""
    assert is_cut(B, T, H)
    q, k, v, d, b, n = inputs(B, T, 1, H, T, lo=1e-3)
    check((q, k, v, most * d, b), n(B, H, D, D).bfloat16(), in_place=in_place)


@pytest.mark.parametrize("lens", [[700, 0, 1, 333], [10] * 60 + [900], [257, 255, 600], [0, 640, 0, 640, 0], [63, 1, 1000, 2]], ids=str)
@pytest.mark.parametrize("in_place", [False, True])
def test_bf16_states_packed(lens, in_place):
    cu = offsets(lens)
    assert is_cut(1, cu[-1], 2, len(lens))
    args = inputs(1, cu[-1], 1, 2, len(lens), lo=1e-4)
    check(args, args[-1](len(lens), 2, D, D).bfloat16(), cu, in_place=in_place)


def check_bwd(args, h0, dht, cu=None):
    q, k, v, decay, beta, n = args
    dout = n(*v.shape).bfloat16()
    c = None if cu is None else torch.tensor(cu, dtype=torch.int64, device=q.device)
    r = gdn.bwd(q, k, v, decay, beta, SCALE, dout, h0, dht, c)
    close_grads(r, gdn_ref_bwd(q, k, v, decay, beta, SCALE, dout, h0, dht, cu))


@pytest.mark.parametrize("B,T,Hk,H", [(1, 1024, 1, 2), (2, 1500, 1, 1), (1, 2049, 1, 3)])
def test_backward_from_bf16_states(B, T, Hk, H):
    assert is_cut(B, T, H)
    args = inputs(B, T, Hk, H, T, lo=1e-4)
    n = args[-1]
    check_bwd(args, n(B, H, D, D).bfloat16(), n(B, H, D, D))


@pytest.mark.parametrize("lens", [[700, 0, 1, 333], [10] * 60 + [900], [0, 640, 0, 640, 0]], ids=str)
def test_backward_from_bf16_states_packed(lens):
    cu = offsets(lens)
    args = inputs(1, cu[-1], 1, 2, len(lens), lo=1e-4)
    n = args[-1]
    check_bwd(args, n(len(lens), 2, D, D).bfloat16(), n(len(lens), 2, D, D), cu)


BAD = [[0, 600, 500, 1500], [1, 5, 700, 1500], [0, 5, 700, 1501], [0, -1, 700, 1500], [0, 1 << 40, 700, 1500], [0, 1600, 1500, 1500]]


@pytest.mark.parametrize("cu", BAD, ids=str)
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T,H", [(1500, 2), (8200, 65)])   # 65 heads: segments long enough that heads are put in an order first
def test_bad_lengths(cu, in_place, T, H):
    """Found on the device: every sequence counts as empty, states pass, nothing else is written."""
    cu = cu[:-1] + [cu[-1] + T - 1500]
    assert is_cut(1, T, H, 3)
    q, k, v, d, b, n = inputs(1, T, 1, H, 9)
    h0 = n(3, H, D, D)
    out = torch.full(v.shape, 7.0, dtype=torch.bfloat16, device=q.device)
    ht = h0.clone() if in_place else torch.full_like(h0, float("nan"))
    ws = gdn.fwd(q, k, v, d, b, SCALE, out, ht if in_place else h0, ht, torch.tensor(cu, device=q.device))
    assert gdn.device_status(ws) != 0
    assert torch.equal(ht, h0) and (out == 7.0).all()


@pytest.mark.parametrize("cu", BAD, ids=str)
@pytest.mark.parametrize("dht", [False, True])
@pytest.mark.parametrize("T,H", [(1500, 2), (8200, 65)])
def test_bad_lengths_backward(cu, dht, T, H):
    cu = cu[:-1] + [cu[-1] + T - 1500]
    q, k, v, d, b, n = inputs(1, T, 1, H, 9)
    h0, dht = n(3, H, D, D), n(3, H, D, D) if dht else None
    r = gdn.bwd(q, k, v, d, b, SCALE, torch.ones_like(v), h0, dht, torch.tensor(cu, device=q.device))
    assert gdn.device_status(r["workspace"]) != 0
    assert torch.equal(r["dinitial_state"], torch.zeros_like(h0) if dht is None else dht)


@pytest.mark.parametrize("decay", [-0.001, -0.3, -5.0])
@pytest.mark.parametrize("name", ["k", "v"])
@pytest.mark.parametrize("packed", [False, True])
def test_key_or_value_that_is_not_finite(name, decay, packed):
    """It reaches its own sequence and head alone, from the first token of its chunk of 32 on; over cuts it lasts where the state does and
    may be forgotten where transitions below 2^-150 lie behind it."""
    cu = [0, 1900, 2500] if packed else None
    q, k, v, d, b, n = inputs(1, 2500, 2, 2, 33)
    assert is_cut(1, 2500, 2, 2 if packed else 0)
    d = torch.full_like(d, decay)
    h0 = n(2 if packed else 1, 2, D, D)
    clean, cfin = run(q, k, v, d, b, h0, cu)
    at, end = 700, 1900 if packed else 2500
    (k if name == "k" else v)[0, at, 1, 7] = float("nan")
    out, fin = run(q, k, v, d, b, h0, cu)
    first = at // 32 * 32
    assert torch.equal(out[:, :, 0], clean[:, :, 0]) and torch.equal(fin[:, 0], cfin[:, 0])
    assert torch.equal(out[:, :first, 1], clean[:, :first, 1])
    if packed:
        assert torch.equal(out[:, end:], clean[:, end:]) and torch.equal(fin[1], cfin[1])
    rest = [i for i in range(D) if i != 7]
    if name == "v":   # its value channel alone
        assert torch.equal(out[:, :, 1, rest], clean[:, :, 1, rest]) and torch.equal(fin[0, 1, rest], cfin[0, 1, rest])
        assert out[0, at, 1, 7].isnan()
    else:
        assert out[0, at, 1].isnan().all()
    if decay == -0.001:   # the state's norm falls by 2.6 from there on at the most: nothing is forgotten
        assert out[0, at:end, 1, 7].isnan().all() and fin[0, 1, 7].isnan().all()
        if name == "k":
            assert out[0, at:end, 1].isnan().all() and fin[0, 1].isnan().all()


@pytest.mark.parametrize("T", [150, 1500])
@pytest.mark.parametrize("name", ["q", "k", "v", "dout"])
@pytest.mark.parametrize("packed", [False, True])
def test_backward_of_values_that_are_not_finite(name, T, packed):
    """They reach the gradients of their own sequence alone, of v and dout those of their own value head (dq and dk are sums over the
    heads that share a q/k head)."""
    q, k, v, d, b, n = inputs(1 if packed else 2, 2 * T if packed else T, 2, 4, 35)
    cu = torch.tensor([0, T, 2 * T], device=q.device) if packed else None
    dout, h0, dht = n(*v.shape).bfloat16(), n(2, 4, D, D), n(2, 4, D, D)
    clean = gdn.bwd(q, k, v, d, b, SCALE, dout, h0, dht, cu)
    x = {"q": q, "k": k, "v": v, "dout": dout}[name]
    at, head = T // 2 + 3, 0 if name in ("q", "k") else 1   # value heads 0 and 1 read q/k head 0
    x[0, at, head, 5] = float("nan")
    r = gdn.bwd(q, k, v, d, b, SCALE, dout, h0, dht, cu)
    per_token = {m: (r[m][0].split(T) if packed else r[m].unbind(0), clean[m][0].split(T) if packed else clean[m].unbind(0))
                 for m in ("dq", "dk", "dv", "ddecay", "dbeta")}
    hit = (0, 1) if name in ("q", "k") else (1,)
    for m, (got, want) in per_token.items():
        assert torch.equal(got[1], want[1]), m
        for h in range(got[0].shape[1]):
            if h not in ((0,) if m in ("dq", "dk") else hit):
                assert torch.equal(got[0][:, h], want[0][:, h]), (m, h)
    assert torch.equal(r["dinitial_state"][1], clean["dinitial_state"][1])
    for h in set(range(4)) - set(hit):
        assert torch.equal(r["dinitial_state"][0, h], clean["dinitial_state"][0, h])
    # where the token's own gradients depend on it
    own = {"q": ("ddecay",), "k": ("dk", "ddecay", "dbeta"), "v": ("dbeta", "dk"), "dout": ("dq", "dv", "ddecay", "dbeta")}[name]
    for m in own:
        y = per_token[m][0][0][at, 0 if m in ("dq", "dk") else hit[0]]
        assert y.isnan().any(), m
