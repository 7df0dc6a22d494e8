"""kda_gdn_fwd and kda_gdn_fwd_recurrent against the 64-bit recurrence, on the GPU."""
import pytest
import torch

from gated_delta_rule_86_amd import gdn

from gdn_testutil import D, close_bf16, close_fp32, close_state, gdn_ref, inputs

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


def run(q, k, v, decay, beta, h0=None, cu=None, call=gdn.fwd, final="fp32", in_place=False, scale=SCALE, **kw):
    N = q.shape[0] if cu is None else len(cu) - 1
    H = v.shape[2]
    out = torch.full(v.shape, float("nan"), dtype=torch.bfloat16, device=q.device)
    dt = h0.dtype if h0 is not None else {"fp32": torch.float32, "bf16": torch.bfloat16}[final]
    if in_place:
        h0 = ht = h0.clone()
    else:
        ht = torch.full((N, H, D, D), float("nan"), dtype=dt, device=q.device)
    c = None if cu is None else torch.tensor(cu, dtype=torch.int64, device=q.device)
    call(q, k, v, decay, beta, scale, out, h0, ht, c, **kw)
    torch.cuda.synchronize()
    return out, ht


def check(args, h0=None, cu=None, what="", grow=1.0, **kw):
    q, k, v, decay, beta = args[:5]
    want, wfin = gdn_ref(q, k, v, decay, beta, SCALE, h0, cu)
    out, fin = run(q, k, v, decay, beta, h0, cu, **kw)
    close_bf16(out, want, (what, "out"), grow)
    close_state(fin, wfin, (what, "final"), grow)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200])
@pytest.mark.parametrize("call", [gdn.fwd, gdn.fwd_recurrent], ids=["chunked", "recurrent"])
def test_lengths(T, call):
    args = inputs(2, T, 2, 2, T)
    h0 = args[-1](2, 2, D, D)
    check(args, h0, call=call)
    check(args, None, call=call)


@pytest.mark.parametrize("Hk,H", [(1, 1), (1, 3), (2, 4), (3, 3), (2, 8)])
@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("call", [gdn.fwd, gdn.fwd_recurrent], ids=["chunked", "recurrent"])
def test_heads_and_strides(Hk, H, strided, call):
    args = inputs(2, 97, Hk, H, 7 * H + Hk, strided=strided)
    check(args, args[-1](2, H, D, D), call=call)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("call", [gdn.fwd, gdn.fwd_recurrent], ids=["chunked", "recurrent"])
def test_state_types(dt, in_place, call):
    args = inputs(3, 70, 2, 2, 5)
    check(args, args[-1](3, 2, D, D).to(dt), call=call, in_place=in_place)


@pytest.mark.parametrize("lens", [[1], [5, 0, 64, 1, 63], [0, 0, 130], [64, 64], [65, 0], [0], [200, 3, 128, 0, 1, 90]], ids=str)
@pytest.mark.parametrize("call", [gdn.fwd, gdn.fwd_recurrent], ids=["chunked", "recurrent"])
@pytest.mark.parametrize("in_place", [False, True])
def test_packed(lens, call, in_place):
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    args = inputs(1, cu[-1], 1, 2, len(lens))
    h0 = args[-1](len(lens), 2, D, D)
    check(args, h0, cu, call=call, in_place=in_place)


@pytest.mark.parametrize("B,T,H", [(1, 1024, 2), (2, 1500, 1), (1, 2049, 3)])
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_cut_into_segments(B, T, H, in_place):
    assert gdn.workspace_size(B, T, H) > 512 + (B * T // 32 + B + 1) * H * 13312  # states of the cuts behind the records
    args = inputs(B, T, 1, H, T, lo=1e-4)
    check(args, args[-1](B, H, D, D), in_place=in_place)
    if not in_place:
        check(args, None)


@pytest.mark.parametrize("lens", [[700, 0, 1, 333], [1500], [10] * 60 + [900], [256, 256, 256, 256], [257, 255, 600],
                                  [0, 640, 0, 640, 0], [63, 1, 1000, 2]], ids=str)
@pytest.mark.parametrize("in_place", [False, True])
def test_packed_and_cut(lens, in_place):
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    args = inputs(1, cu[-1], 1, 2, len(lens), lo=1e-4)
    h0 = args[-1](len(lens), 2, D, D)
    check(args, h0, cu, in_place=in_place)


@pytest.mark.parametrize("keys", ["normal", "same"])
@pytest.mark.parametrize("beta", [0.0, 1.0, 2.0])
@pytest.mark.parametrize("decay", [0.0, -0.01, -20.0, -1000.0, float("-inf")])
def test_gates(keys, beta, decay):
    """beta 0 writes nothing, beta 1 replaces, beta 2 reflects; no decay, and decays that forget."""
    q, k, v, d, b, n = inputs(1, 150, 1, 2, 3, keys=keys)
    d = torch.full_like(d, decay)
    b = torch.full_like(b, beta)
    if decay == -1000.0:
        d[:, ::7] = 0.0
    # With beta 2 and one key for all tokens, S k -> 2 v - S k: nothing damps an error, and those of T = 150 tokens add up
    # like a walk, to sqrt(150) = 12 times one token's, where decays or beta < 2 keep them near one.
    check((q, k, v, d, b), n(1, 2, D, D), grow=12.0 if beta == 2.0 else 1.0)


def test_mixed_gates():
    """Forgetting in the middle of chunks next to slow decays, positive decays counted as 0, zero keys and queries."""
    q, k, v, d, b, n = inputs(2, 190, 2, 2, 11, lo=1e-6)
    d[:, 40:50] = -1000.0
    d[:, 100] = float("-inf")
    d[:, 120:130] = 0.5
    d[0, 64:128] = -30.0
    b[:, 60:70] = 0.0
    k[:, 30:34] = 0.0
    q[:, 80:90] = 0.0
    check((q, k, v, d, b), n(2, 2, D, D))


def test_paths_agree_and_repeat():
    """The chunked form, token by token and cut sequences agree; a second run gives the same bits."""
    args = inputs(1, 1300, 1, 2, 17)
    q, k, v, d, b, n = args
    h0 = n(1, 2, D, D)
    o1, f1 = run(q, k, v, d, b, h0)
    o2, f2 = run(q, k, v, d, b, h0)
    assert torch.equal(o1, o2) and torch.equal(f1, f2)
    o3, f3 = run(q, k, v, d, b, h0, call=gdn.fwd_recurrent)
    close_fp32(f1, f3, "final")
    close_bf16(o1, gdn_ref(q, k, v, d, b, SCALE, h0)[0], "out")
    close_bf16(o3, gdn_ref(q, k, v, d, b, SCALE, h0)[0], "out")


def test_out_without_states():
    args = inputs(1, 100, 1, 1, 4)
    q, k, v, d, b, _ = args
    out = torch.empty_like(v)
    assert gdn.fwd_recurrent(q, k, v, d, b, SCALE, out) is None
    want = gdn_ref(q, k, v, d, b, SCALE)[0]
    close_bf16(out, want, "recurrent")
    out.fill_(float("nan"))
    gdn.fwd(q, k, v, d, b, SCALE, out)
    close_bf16(out, want, "chunked")


@pytest.mark.parametrize("call", [gdn.fwd, gdn.fwd_recurrent], ids=["chunked", "recurrent"])
@pytest.mark.parametrize("cu", [[0, 5, 4, 20], [1, 5, 10, 20], [0, 5, 10, 21]], ids=str)
def test_bad_lengths_make_every_sequence_empty(call, cu):
    q, k, v, d, b, n = inputs(1, 20, 1, 2, 9)
    h0 = n(3, 2, D, D)
    out = torch.full(v.shape, 7.0, dtype=torch.bfloat16, device=q.device)
    ht = torch.full_like(h0, float("nan"))
    ws = call(q, k, v, d, b, SCALE, out, h0, ht, torch.tensor(cu, device=q.device))
    assert gdn.device_status(ws) != 0
    assert torch.equal(ht, h0) and (out == 7.0).all()


@pytest.mark.parametrize("T", [0])
def test_no_tokens(T):
    q, k, v, d, b, n = inputs(2, 0, 1, 2, 9)
    h0 = n(2, 2, D, D)
    for call in (gdn.fwd, gdn.fwd_recurrent):
        out, ht = run(q, k, v, d, b, h0, call=call)
        assert torch.equal(ht, h0)


def test_not_finite_stays_in_its_head():
    """A NaN value, an infinite key and a NaN gate reach their own sequence and head alone, behind the chunk's first token."""
    q, k, v, d, b, n = inputs(2, 300, 3, 3, 21)
    h0 = n(2, 3, D, D)
    clean, cfin = run(q, k, v, d, b, h0)
    v[0, 100, 0, 5] = float("nan")
    k[1, 130, 1, 3] = float("inf")
    d[0, 200, 2] = float("nan")
    for call in (gdn.fwd, gdn.fwd_recurrent):
        out, fin = run(q, k, v, d, b, h0, call=call)
        ref, rfin = (clean, cfin) if call is gdn.fwd else run(*[x.nan_to_num(0, 0, 0) for x in (q, k, v, d, b)], h0, call=call)
        for bi, h in ((1, 0), (0, 1), (1, 2)):
            assert torch.equal(out[bi, :, h], ref[bi, :, h]) and torch.equal(fin[bi, h], rfin[bi, h])
        assert torch.equal(out[0, :64, 0], ref[0, :64, 0]) and torch.equal(out[1, :128, 1], ref[1, :128, 1])
        assert torch.equal(out[0, :192, 2], ref[0, :192, 2])
        assert out[0, 100, 0].isnan().any() and out[1, 130, 1].isnan().any() and out[0, 200:, 2].isnan().all()


@pytest.mark.parametrize("lo,hi", [(0.05, 0.5), (1.0, 20.0), (0.0, 3.0)], ids=str)
@pytest.mark.parametrize("beta", [0.9, 2.5])
@pytest.mark.parametrize("in_place", [False, True])
def test_cut_rows_that_forget(lo, hi, beta, in_place):
    """Decays that leave nothing of a state behind a few hundred tokens, a few, or in one head only: what the cuts leave out counts
    as 0.  beta 2.5 makes single transitions grow."""
    q, k, v, d, b, n = inputs(1, 3000, 1, 3, 31)
    d = -(lo + (hi - lo) * torch.rand(d.shape, device=d.device))
    d[:, :, 2] *= 1e-3
    b = b * beta
    if beta > 2:  # no running away in the head that keeps its state
        b[:, :, 2] *= 0.3
    check((q, k, v, d, b), n(1, 3, D, D), in_place=in_place)
    cu = [0, 1300, 1301, 3000]
    check((q, k, v, d, b), n(3, 3, D, D), cu, in_place=in_place)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("decay", [-0.001, -5.0])
def test_state_that_is_not_finite_lasts(bad, decay):
    """A row of the initial state that is not finite stays NaN to the end, over cuts of its sequence too, and reaches nothing else."""
    q, k, v, d, b, n = inputs(1, 2500, 1, 2, 33)
    d = torch.full_like(d, decay)
    h0 = n(1, 2, D, D)
    clean, cfin = run(q, k, v, d, b, h0)
    h0[0, 1, 7, 9] = bad
    out, fin = run(q, k, v, d, b, h0)
    keep = torch.ones(D, dtype=torch.bool, device=q.device)
    keep[7] = False
    assert torch.equal(out[:, :, 0], clean[:, :, 0]) and torch.equal(out[:, :, 1, keep], clean[:, :, 1, keep])
    assert torch.equal(fin[:, 0], cfin[:, 0]) and torch.equal(fin[:, 1, keep], cfin[:, 1, keep])
    assert fin[0, 1, 7].isnan().all() and not torch.isfinite(out[:, :, 1, 7]).any()
