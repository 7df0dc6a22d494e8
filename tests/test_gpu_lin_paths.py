"""Paths of the decayed linear attention that depend on what is asked for: the backward pass without the decay's gradient over cut and
packed rows, rows without tokens, a bf16 final state without an initial one, cu_seqlens_host."""
import pytest
import torch

from gated_delta_rule_86_amd import linattn
from gated_delta_rule_86_amd.kda import KDAError
from lin_testutil import D, close_bf16, close_fp32, dev, inputs, lin_ref, lin_ref_chunked
from test_gpu_linattn import CUS, bwd_ref, check_bwd, states

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


@pytest.mark.parametrize("need_ddecay", [False, True])
@pytest.mark.parametrize("Hk,H", [(1, 3), (2, 2)])
@pytest.mark.parametrize("h0_dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("cu", CUS + [[0, 2000, 2001, 5000]], ids=str)
def test_backward_packed(cu, h0_dtype, Hk, H, need_ddecay):
    T, N = cu[-1], len(cu) - 1
    assert (linattn.bwd_workspace_size(1, T, H, H, N, True, False) > 256) == (T > 1000)  # slots: the row is cut
    q, k, v, d, n = inputs(1, T, Hk, H, 17 + N, "head", strided=True)
    h0, dht, do = states(N, H, h0_dtype, n), n(N, H, D, D), n(1, T, H, D).bfloat16()
    r = linattn.bwd(q, k, v, d, SCALE, do, h0, dht, torch.tensor(cu, device=dev()), need_ddecay=need_ddecay)
    assert ("ddecay" in r) == need_ddecay
    check_bwd(r, bwd_ref(q, k, v, d, do, h0, dht, cu), q, k, d)


@pytest.mark.parametrize("need_ddecay", [False, True])
@pytest.mark.parametrize("B,T,Hk,H,decay", [(1, 4096, 2, 2, "token"), (2, 3001, 1, 2, "head"), (1, 2500, 1, 4, "token")])
def test_backward_cut(B, T, Hk, H, decay, need_ddecay):
    q, k, v, d, n = inputs(B, T, Hk, H, T, decay, lo=1e-4)
    h0, dht, do = states(B, H, torch.float32, n), n(B, H, D, D), n(B, T, H, D).bfloat16()
    r = linattn.bwd(q, k, v, d, SCALE, do, h0, dht, need_ddecay=need_ddecay)
    check_bwd(r, bwd_ref(q, k, v, d, do, h0, dht, None), q, k, d)
    r = linattn.bwd(q, k, v, d, SCALE, do, None, None, need_ddecay=need_ddecay)
    check_bwd(r, bwd_ref(q, k, v, d, do, None, None, None), q, k, d)


@pytest.mark.parametrize("f", [linattn.fwd, linattn.fwd_recurrent])
@pytest.mark.parametrize("decay", ["head", "token"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_rows_without_tokens(f, decay, dtype):
    """T = 0 without cu_seqlens: final states are the initial ones (0 without), and their gradients pass through."""
    q, k, v, d, n = inputs(3, 0, 2, 4, 1, decay)
    h0, out = states(3, 4, dtype, n), torch.empty_like(v)
    ht = torch.full_like(h0, 7.0)
    f(q, k, v, d, SCALE, out, h0, ht)
    assert torch.equal(ht, h0)
    f(q, k, v, d, SCALE, out, None, ht)
    assert (ht == 0).all()
    same = h0.clone()
    f(q, k, v, d, SCALE, out, same, same)
    assert torch.equal(same, h0)
    dht = n(3, 4, D, D)
    for g in (dht, None):
        r = linattn.bwd(q, k, v, d, SCALE, out, h0, g)
        assert torch.equal(r["dinitial_state"], torch.zeros_like(dht) if g is None else g)
        assert (r["ddecay"] == 0).all() and r["dq"].shape == q.shape and r["dv"].shape == v.shape


@pytest.mark.parametrize("T", [1, 70, 2500])
@pytest.mark.parametrize("packed", [False, True])
def test_bf16_final_state_without_an_initial_one(T, packed):
    q, k, v, d, n = inputs(1, T, 1, 2, T, "token")
    cu = [0, T // 3, T] if packed else None
    ro, rs = lin_ref_chunked(q, k, v, d, SCALE, None, cu)
    c = None if cu is None else torch.tensor(cu, device=dev())
    for f in (linattn.fwd, linattn.fwd_recurrent):
        out, ht = torch.empty_like(v), torch.empty(rs.shape, dtype=torch.bfloat16, device=dev())
        f(q, k, v, d, SCALE, out, None, ht, c)
        close_bf16(out, ro, "out")
        close_bf16(ht, rs, "final")


def test_cu_seqlens_host():
    """The host copy changes no result, and a bad one is refused before any launch."""
    cu = [0, 700, 700, 1400, 2000]
    q, k, v, d, n = inputs(1, 2000, 1, 2, 3, "token")
    h0, do, dht = states(4, 2, torch.float32, n), n(1, 2000, 2, D).bfloat16(), n(4, 2, D, D)
    c = torch.tensor(cu, device=dev())
    got = []
    for host in (None, cu, torch.tensor(cu)):
        for f in (linattn.fwd, linattn.fwd_recurrent):
            out, ht = torch.empty_like(v), torch.empty_like(h0)
            f(q, k, v, d, SCALE, out, h0, ht, c, cu_seqlens_host=host)
            got += [out, ht]
        r = linattn.bwd(q, k, v, d, SCALE, do, h0, dht, c, cu_seqlens_host=host)
        got += [r[m] for m in ("dq", "dk", "dv", "ddecay", "dinitial_state")]
    third = len(got) // 3
    assert all(torch.equal(a, b) for a, b in zip(got[third:], got[:third] * 2))
    close_bf16(got[0], lin_ref(q, k, v, d, SCALE, h0, cu)[0], "out")
    close_fp32(got[1], lin_ref(q, k, v, d, SCALE, h0, cu)[1], "final")
    out = torch.full_like(v, 7.0)
    for bad in ([1, 700, 700, 1400, 2000], [0, 700, 600, 1400, 2000], [0, 700, 700, 1400, 1999]):
        for f in (linattn.fwd, linattn.fwd_recurrent):
            with pytest.raises(KDAError, match="CU_SEQLENS"):
                f(q, k, v, d, SCALE, out, h0, None, c, cu_seqlens_host=bad)
        with pytest.raises(KDAError, match="CU_SEQLENS"):
            linattn.bwd(q, k, v, d, SCALE, do, h0, dht, c, cu_seqlens_host=bad)
    torch.cuda.synchronize()
    assert (out == 7.0).all()


def test_token_by_token_up_to_its_limit():
    """As many sequences x heads as a launch holds, without states: out = scale (q.k) v."""
    B, H = (1 << 22) - 2, 4
    q, k, v, d, _ = inputs(B, 1, 1, H, 5, "token")
    out = torch.empty_like(v)
    linattn.fwd_recurrent(q, k, v, d, SCALE, out)
    for at in (slice(0, 1000), slice(B // 2, B // 2 + 1000), slice(B - 1000, B)):
        close_bf16(out[at], SCALE * (q[at].double() * k[at].double()).sum(-1, keepdim=True) * v[at].double(), "out")


@pytest.mark.parametrize("cu", [None, [0, 64, 64, 900], [0, 1300, 2600]], ids=str)
@pytest.mark.parametrize("need_ddecay", [False, True])
def test_backward_without_the_initial_states_gradient(cu, need_ddecay):
    """Not allocated, not written; everything else keeps its bits."""
    T, N = 200 if cu is None else cu[-1], 1 if cu is None else len(cu) - 1
    q, k, v, d, n = inputs(1, T, 1, 2, T, "token")
    dht, do = n(N, 2, D, D), n(1, T, 2, D).bfloat16()
    c = None if cu is None else torch.tensor(cu, device=dev())
    a = linattn.bwd(q, k, v, d, SCALE, do, None, dht, c, need_ddecay=need_ddecay)
    b = linattn.bwd(q, k, v, d, SCALE, do, None, dht, c, need_ddecay=need_ddecay, need_dinitial_state=False)
    assert set(a) - set(b) == {"dinitial_state"}
    assert all(torch.equal(a[m], b[m]) for m in set(b) - {"workspace"})
