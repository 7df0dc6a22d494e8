"""Decayed linear attention (kda_lin_fwd, kda_lin_fwd_recurrent, kda_lin_bwd) against plain 64-bit references."""
import pytest
import torch

from gated_delta_rule_86_amd import linattn
from lin_testutil import D, close_bf16, close_ddecay, close_fp32, dev, inputs, lin_ref, lin_ref_chunked

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


def states(n_seq, H, dtype, n):
    return None if dtype is None else (0.5 * n(n_seq, H, D, D)).to(dtype)


def run_fwd(q, k, v, d, h0, cu, dtype=torch.float32, recurrent=False, in_place=False, **kw):
    B, T, H = v.shape[:3]
    N = B if cu is None else len(cu) - 1
    out = torch.full((B, T, H, D), float("nan"), dtype=torch.bfloat16, device=dev())
    ht = h0 if in_place else torch.full((N, H, D, D), float("nan"), dtype=dtype, device=dev())
    c = None if cu is None else torch.tensor(cu, dtype=torch.int64, device=dev())
    (linattn.fwd_recurrent if recurrent else linattn.fwd)(q, k, v, d, SCALE, out, h0, ht, c, **kw)
    torch.cuda.synchronize()
    return out, ht


def check_state(got, want, dtype, what):
    if dtype == torch.bfloat16:
        close_bf16(got, want, what)
    else:
        close_fp32(got, want, what)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200])
@pytest.mark.parametrize("decay", ["head", "token"])
@pytest.mark.parametrize("recurrent", [False, True])
def test_forward_lengths(T, decay, recurrent):
    q, k, v, d, n = inputs(2, T, 2, 4, 100 + T, decay)
    h0 = states(2, 4, torch.float32, n)
    out, ht = run_fwd(q, k, v, d, h0, None, recurrent=recurrent)
    ro, rs = lin_ref(q, k, v, d, SCALE, h0)
    close_bf16(out, ro, "out")
    close_fp32(ht, rs, "final")


CUS = [[0, 5], [0, 1, 2, 3], [0, 0, 70, 70, 70, 131, 131], [0, 64, 128, 129, 400], [0, 300, 301, 700, 701, 1100],
       [0, 0], [0, 513, 513, 1029]]


@pytest.mark.parametrize("cu", CUS, ids=str)
@pytest.mark.parametrize("dtype", [None, torch.bfloat16, torch.float32], ids=str)
def test_forward_varlen(cu, dtype):
    q, k, v, d, n = inputs(1, cu[-1], 1, 3, 7 + len(cu), "token", strided=True)
    h0 = states(len(cu) - 1, 3, dtype, n)
    for recurrent in (False, True):
        out, ht = run_fwd(q, k, v, d, h0, cu, dtype or torch.float32, recurrent)
        ro, rs = lin_ref(q, k, v, d, SCALE, h0, cu)
        close_bf16(out, ro, "out")
        check_state(ht, rs, dtype, "final")


@pytest.mark.parametrize("B,T,Hk,H,decay", [(1, 4096, 1, 1, "head"), (1, 5000, 2, 4, "token"), (3, 1111, 1, 2, "token"),
                                            (2, 2048, 4, 4, "head")])
def test_forward_cut_rows(B, T, Hk, H, decay):
    """Long rows with few heads: segments, states pass, scan; slow decays carry over many segments."""
    assert linattn.workspace_size(B, T, H) > 65536
    q, k, v, d, n = inputs(B, T, Hk, H, 40 + T, decay, lo=1e-5)
    h0 = states(B, H, torch.float32, n)
    out, ht = run_fwd(q, k, v, d, h0, None)
    ro, rs = lin_ref_chunked(q, k, v, d, SCALE, h0)
    close_bf16(out, ro, "out")
    close_fp32(ht, rs, "final")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("cu", [None, [0, 700, 700, 1400, 1401, 4000]], ids=["rows", "varlen"])
def test_state_in_place(dtype, cu):
    """initial_state = final_state with cut rows: the same bits as with separate buffers."""
    q, k, v, d, n = inputs(1, 4000, 1, 2, 5, "token")
    h0 = states(1 if cu is None else len(cu) - 1, 2, dtype, n)
    for recurrent in (False, True):
        out, ht = run_fwd(q, k, v, d, h0, cu, dtype, recurrent)
        h1 = h0.clone()
        o1, s1 = run_fwd(q, k, v, d, h1, cu, dtype, recurrent, in_place=True)
        assert s1 is h1 and torch.equal(o1, out) and torch.equal(s1, ht)


def bwd_ref(q, k, v, d, do, h0, dht, cu, chunked=True):
    leaf = lambda x: None if x is None else x.detach().double().contiguous().requires_grad_()  # noqa: E731
    ql, kl, vl, dl, hl = leaf(q), leaf(k), leaf(v), leaf(d), leaf(h0)
    if hl is None:
        N = q.shape[0] if cu is None else len(cu) - 1
        hl = torch.zeros(N, v.shape[2], D, D, dtype=torch.float64, device=q.device, requires_grad=True)
    o, s = (lin_ref_chunked if chunked else lin_ref)(ql, kl, vl, dl, SCALE, hl, cu)
    loss = (o * do.double()).sum()
    if dht is not None:
        loss = loss + (s * dht.double()).sum()
    g = torch.autograd.grad(loss, (ql, kl, vl, dl, hl), allow_unused=True)
    r = dict(zip(("dq", "dk", "dv", "ddecay", "dinitial_state"),
                 (torch.zeros_like(x) if y is None else y for x, y in zip((ql, kl, vl, dl, hl), g))))
    return r | {"final": s.detach(), "dfinal": dht}


def check_bwd(r, ref, q, k, d):
    for n in ("dq", "dk", "dv"):
        close_bf16(r[n], ref[n], n)
    close_fp32(r["dinitial_state"], ref["dinitial_state"], "dinitial_state")
    if "ddecay" in r:
        close_ddecay(r["ddecay"], ref["ddecay"], q, ref["dq"], k, ref["dk"], d, ref["final"], ref["dfinal"])


@pytest.mark.parametrize("T", [1, 2, 17, 32, 33, 64, 65, 130])
@pytest.mark.parametrize("decay,Hk,H", [("head", 2, 2), ("token", 2, 4), ("head", 1, 3)])
def test_backward_lengths(T, decay, Hk, H):
    q, k, v, d, n = inputs(2, T, Hk, H, 300 + T, decay, strided=True)
    h0, dht = states(2, H, torch.float32, n), n(2, H, D, D)
    do = n(2, T, H, D).bfloat16()
    r = linattn.bwd(q, k, v, d, SCALE, do, h0, dht)
    check_bwd(r, bwd_ref(q, k, v, d, do, h0, dht, None, chunked=T > 33), q, k, d)
    r2 = linattn.bwd(q, k, v, d, SCALE, do, None, None, need_ddecay=False)
    assert "ddecay" not in r2
    check_bwd(r2, bwd_ref(q, k, v, d, do, None, None, None), q, k, d)


@pytest.mark.parametrize("cu", CUS + [[0, 2000, 2001, 5000]], ids=str)
@pytest.mark.parametrize("decay", ["head", "token"])
def test_backward_varlen(cu, decay):
    q, k, v, d, n = inputs(1, cu[-1], 1, 2, 17 + len(cu), decay)
    N = len(cu) - 1
    h0, dht = states(N, 2, torch.bfloat16, n), n(N, 2, D, D)
    do = n(1, cu[-1], 2, D).bfloat16()
    c = torch.tensor(cu, dtype=torch.int64, device=dev())
    r = linattn.bwd(q, k, v, d, SCALE, do, h0, dht, c)
    check_bwd(r, bwd_ref(q, k, v, d, do, h0, dht, cu), q, k, d)


@pytest.mark.parametrize("B,T,Hk,H,decay", [(1, 4096, 2, 2, "token"), (2, 3001, 1, 2, "head")])
def test_backward_cut_rows(B, T, Hk, H, decay):
    q, k, v, d, n = inputs(B, T, Hk, H, T, decay, lo=1e-4)
    h0, dht = states(B, H, torch.float32, n), n(B, H, D, D)
    do = n(B, T, H, D).bfloat16()
    r = linattn.bwd(q, k, v, d, SCALE, do, h0, dht)
    check_bwd(r, bwd_ref(q, k, v, d, do, h0, dht, None), q, k, d)


def test_backward_differences():
    """Gradients against central differences of the fp64 recurrence in random directions."""
    q, k, v, d, n = inputs(1, 40, 1, 2, 9, "token")
    h0, dht = states(1, 2, torch.float32, n), n(1, 2, D, D)
    do = n(1, 40, 2, D).bfloat16()
    r = linattn.bwd(q, k, v, d, SCALE, do, h0, dht)

    def loss(*a):
        o, s = lin_ref(*a[:4], SCALE, a[4])
        return float((o * do.double()).sum() + (s * dht.double()).sum())
    args = [x.double() for x in (q, k, v, d, h0)]
    for i, name in enumerate(("dq", "dk", "dv", "ddecay", "dinitial_state")):
        u = n(*args[i].shape).double() * (1e-3 if name == "ddecay" else 1.0)
        step = 1e-4 if name != "ddecay" else 1e-2
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + step * u, args[i] - step * u
        want = (loss(*hi) - loss(*lo)) / (2 * step)
        got = float((r[name].double() * u).sum())
        # |g . u| for independent errors of 2^-8 in g: 2^-8 |g| |u| / sqrt(numel) per direction, five times that
        tol = 5 * 2.0 ** -8 * float(r[name].double().norm() * u.norm()) / u.numel() ** 0.5 + 1e-6 * abs(want)
        assert abs(got - want) <= tol, (name, got, want, tol)


def test_extreme_decays():
    """0 keeps everything, -inf forgets, values above 0 count as 0; several resets in a chunk stay exact."""
    q, k, v, d, n = inputs(1, 200, 1, 2, 3, "token")
    d[:, ::7] = float("-inf")
    d[:, 3::5] = 0.0
    d[:, 50:90, 1] = 0.25
    d[:, 100:130] = -1e30
    d[:, 140:150] = -150.0
    h0 = states(1, 2, torch.float32, n)
    ro, rs = lin_ref(q, k, v, d, SCALE, h0)
    for recurrent in (False, True):
        out, ht = run_fwd(q, k, v, d, h0, None, recurrent=recurrent)
        close_bf16(out, ro, "out")
        close_fp32(ht, rs, "final")
    do, dht = n(1, 200, 2, D).bfloat16(), n(1, 2, D, D)
    r = linattn.bwd(q, k, v, d, SCALE, do, h0, dht)
    ref = bwd_ref(q, k, v, d, do, h0, dht, None)
    check_bwd(r, ref, q, k, d)
    off = (d > 0) | (d <= -1000.0)
    assert (r["ddecay"][off] == 0).all()


def test_no_decay_and_slow_decay_over_a_long_row():
    """Decay 0 and -1e-6 over 20000 tokens: factors near 1 must not drift."""
    q, k, v, _, n = inputs(1, 20000, 1, 2, 4, "head")
    d = torch.tensor([0.0, -1e-6], device=dev())
    out, ht = run_fwd(q, k, v, d, None, None)
    ro, rs = lin_ref_chunked(q, k, v, d, SCALE, None, C=500)
    close_bf16(out, ro, "out")
    close_fp32(ht, rs, "final")


def test_neighbours_and_rows_behind():
    """NaN in one sequence and head stays there; memory around out and states is left alone."""
    cu = [0, 100, 165, 300]
    q, k, v, d, n = inputs(1, 300, 2, 2, 8, "token")
    h0 = states(3, 2, torch.float32, n)
    want, wst = run_fwd(q, k, v, d, h0, cu)
    v2 = v.clone()
    v2[0, 120, 1] = float("nan")
    k2 = k.clone()
    k2[0, 130, 1] = float("inf")
    out, ht = run_fwd(q, k2, v2, d, h0, cu)
    assert torch.equal(out[0, :, 0], want[0, :, 0]) and torch.equal(ht[:, 0], wst[:, 0])
    for a, b in ((0, 100), (165, 300)):
        assert torch.equal(out[0, a:b, 1], want[0, a:b, 1])
    assert torch.equal(ht[0, 1], wst[0, 1]) and torch.equal(ht[2, 1], wst[2, 1])
    assert torch.isnan(out[0, 120:165, 1].float()).all()


def test_deterministic_and_workspace_poison():
    q, k, v, d, n = inputs(1, 3000, 1, 2, 21, "token")
    h0, do = states(1, 2, torch.float32, n), n(1, 3000, 2, D).bfloat16()
    dht = n(1, 2, D, D)
    ws = torch.full((linattn.workspace_size(1, 3000, 2),), 255, dtype=torch.uint8, device=dev())
    wb = torch.full((linattn.bwd_workspace_size(1, 3000, 1, 2),), 255, dtype=torch.uint8, device=dev())
    a = run_fwd(q, k, v, d, h0, None)
    b = run_fwd(q, k, v, d, h0, None, workspace=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert linattn.device_status(ws) == 0
    x = linattn.bwd(q, k, v, d, SCALE, do, h0, dht)
    y = linattn.bwd(q, k, v, d, SCALE, do, h0, dht, workspace=wb)
    for m in ("dq", "dk", "dv", "ddecay", "dinitial_state"):
        assert torch.equal(x[m], y[m]), m


def test_invalid_cu_seqlens_on_the_device():
    q, k, v, d, n = inputs(1, 64, 1, 1, 2, "token")
    h0 = states(3, 1, torch.float32, n)
    for cu, bits in (([0, 40, 30, 64], 2), ([1, 2, 3, 64], 1), ([0, 2, 3, 63], 4)):
        for recurrent in (False, True):
            ws = torch.empty(max(256, linattn.workspace_size(1, 64, 1, 3, True)), dtype=torch.uint8, device=dev())
            out, ht = run_fwd(q, k, v, d, h0, cu, recurrent=recurrent, workspace=ws)
            assert linattn.device_status(ws) == bits
            assert torch.isnan(out.float()).all() and torch.equal(ht, h0)
        c = torch.tensor(cu, dtype=torch.int64, device=dev())
        r = linattn.bwd(q, k, v, d[0, 0].contiguous(), SCALE, v.contiguous(), h0, h0, c)
        assert torch.equal(r["dinitial_state"], h0) and (r["ddecay"] == 0).all()


def test_other_stream_and_graph():
    """Captured forward and backward, replayed on changed inputs between eager calls, equal the eager results."""
    q, k, v, d, n = inputs(1, 1500, 1, 2, 33, "token")
    cu = torch.tensor([0, 700, 1500], dtype=torch.int64, device=dev())
    h0, do, dht = states(2, 2, torch.float32, n), n(1, 1500, 2, D).bfloat16(), n(2, 2, D, D)
    out, ht = torch.empty_like(v), torch.empty_like(h0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        linattn.fwd(q, k, v, d, SCALE, out, h0, ht, cu)
        linattn.bwd(q, k, v, d, SCALE, do, h0, dht, cu)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        linattn.fwd(q, k, v, d, SCALE, out, h0, ht, cu)
        r = linattn.bwd(q, k, v, d, SCALE, do, h0, dht, cu)
    for i in range(3):
        v.copy_(n(1, 1500, 2, D).bfloat16())
        d.mul_(0.5)
        o2, h2 = torch.empty_like(v), torch.empty_like(h0)
        linattn.fwd(q, k, v, d, SCALE, o2, h0, h2, cu)
        e = linattn.bwd(q, k, v, d, SCALE, do, h0, dht, cu)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(ht, h2)
        for m in ("dq", "dk", "dv", "ddecay", "dinitial_state"):
            assert torch.equal(r[m], e[m]), (i, m)
    o3 = torch.empty_like(v)
    side.wait_stream(torch.cuda.current_stream())
    linattn.fwd(q, k, v, d, SCALE, o3, h0, None, cu, stream=side)
    side.synchronize()
    assert torch.equal(o3, o2)


def test_extents_of_strided_views():
    """Memory between the rows of the views is neither read into results nor written: NaN all around q, k and v."""
    B, T, H = 2, 130, 2
    q, k, v, d, n = inputs(B, T, H, H, 61, "token")
    wide = torch.full((B, T + 3, 3, H, D + 16), float("nan"), dtype=torch.bfloat16, device=dev())
    views = [wide[:, 1:T + 1, i, :, 8:-8] for i in range(3)]
    for x, y in zip(views, (q, k, v)):
        x.copy_(y)
    h0, do = states(B, H, torch.float32, n), n(B, T, H, D).bfloat16()
    want, ws = run_fwd(q, k, v, d, h0, None)
    out, ht = run_fwd(*views, d, h0, None)
    assert torch.equal(out, want) and torch.equal(ht, ws)
    o2, s2 = run_fwd(*views, d, h0, None, recurrent=True)
    close_bf16(o2, lin_ref(q, k, v, d, SCALE, h0)[0], "out")
    a, b = linattn.bwd(q, k, v, d, SCALE, do, h0), linattn.bwd(*views, d, SCALE, do, h0)
    for m in ("dq", "dk", "dv", "ddecay", "dinitial_state"):
        assert torch.equal(a[m], b[m]), m


def test_broadcast_heads_and_batches():
    """q and k expanded over heads and batch rows (strides 0) read as their copies."""
    q, k, v, d, n = inputs(2, 90, 4, 4, 62, "token")
    q1, k1 = q[:1, :, :1].expand(2, -1, 4, -1), k[:1, :, :1].expand(2, -1, 4, -1)
    a = run_fwd(q1, k1, v, d, None, None)
    b = run_fwd(q1.contiguous(), k1.contiguous(), v, d, None, None)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_streams_at_once():
    """Two calls of different sizes side by side, each with its own workspace, give what they give alone."""
    sets = []
    for i, (T, H) in enumerate([(3000, 2), (700, 8)]):
        q, k, v, d, n = inputs(1, T, 1, H, 70 + i, "token")
        do = n(1, T, H, D).bfloat16()
        sets.append((q, k, v, d, do, run_fwd(q, k, v, d, None, None), linattn.bwd(q, k, v, d, SCALE, do)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = []
        for s, (q, k, v, d, do, _, _) in zip(streams, sets):
            out, ht = torch.empty_like(v), torch.empty(1, v.shape[2], D, D, device=dev())
            s.wait_stream(torch.cuda.current_stream())
            linattn.fwd(q, k, v, d, SCALE, out, None, ht, stream=s)
            got.append((out, ht, linattn.bwd(q, k, v, d, SCALE, do, stream=s)))
        torch.cuda.synchronize()
        for (out, ht, r), (*_, f, b) in zip(got, sets):
            assert torch.equal(out, f[0]) and torch.equal(ht, f[1])
            assert all(torch.equal(r[m], b[m]) for m in ("dq", "dk", "dv", "ddecay"))


def test_many_short_sequences():
    """More sequences than segments, single tokens and empty ones among them, and sequences as long as a segment."""
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 9, (400,), generator=g).tolist() + [256, 0, 257, 1, 255]
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    q, k, v, d, n = inputs(1, cu[-1], 1, 1, 63, "token")
    h0 = states(len(lens), 1, torch.float32, n)
    ro, rs = lin_ref(q, k, v, d, SCALE, h0, cu)
    for recurrent in (False, True):
        out, ht = run_fwd(q, k, v, d, h0, cu, recurrent=recurrent)
        close_bf16(out, ro, "out")
        close_fp32(ht, rs, "final")
    do, dht = n(1, cu[-1], 1, D).bfloat16(), n(len(lens), 1, D, D)
    r = linattn.bwd(q, k, v, d, SCALE, do, h0, dht, torch.tensor(cu, device=dev()))
    check_bwd(r, bwd_ref(q, k, v, d, do, h0, dht, cu, chunked=True), q, k, d)


def test_outputs_past_32_bits():
    """out, dout and dv of more than 2^31 elements.  A reset 100 tokens before the end makes the last tokens a small problem
    of their own, and leaves nothing to the gradients before them."""
    T, H, tail = 131200, 128, 100
    q, k, _, _, n = inputs(1, T, 1, 1, 80)
    v = n(T * (D + 8 * H)).bfloat16().as_strided((1, T, H, D), (0, D + 8 * H, 8, 1))
    d = -0.02 * n(1, T, H).abs()
    d[:, T - tail] = float("-inf")
    last = lambda x: x[:, T - tail:]  # noqa: E731
    out, ht = run_fwd(q, k, v, d, None, None)
    assert out.numel() > 2 ** 31 and torch.isfinite(out[:, ::997]).all()
    ro, rs = lin_ref(last(q), last(k), last(v), last(d), SCALE)
    close_bf16(last(out), ro, "out")
    close_fp32(ht, rs, "final")
    do = out.zero_()
    last(do).copy_(n(1, tail, H, D))
    r = linattn.bwd(q, k, v, d, SCALE, do)
    assert all((r[m][:, :T - tail] == 0).all() for m in ("dq", "dk"))
    assert all((r["dv"][:, i:T - tail:31] == 0).all() for i in (0, 17))
    # ddecay is a sum over the later tokens of its segment, so up to 512 tokens before the reset it is 0 to rounding only
    wide = lambda x: x[:, T - tail - 512:]  # noqa: E731
    assert (r["ddecay"][:, :T - tail - 512] == 0).all()
    ref = bwd_ref(wide(q), wide(k), wide(v), wide(d), wide(do), None, None, None)
    check_bwd({m: wide(r[m]) for m in ("dq", "dk", "dv", "ddecay")} | {"dinitial_state": r["dinitial_state"]}, ref,
              wide(q), wide(k), wide(d))


def test_strides_past_32_bits():
    """Batch rows 2^31 elements apart read as their copies."""
    T, H = 70, 2
    base = torch.empty((1 << 31) + T * 3 * H * D, dtype=torch.bfloat16, device=dev())
    x = base.as_strided((2, T, 3 * H, D), (1 << 31, 3 * H * D, D, 1))
    q, k, v, d, n = inputs(2, T, 3 * H, 3 * H, 81)
    x.copy_(q)
    q, k, v = x.split(H, 2)
    d, do = d[:, :, :H].contiguous(), n(2, T, H, D).bfloat16()
    c = [y.contiguous() for y in (q, k, v)]
    for recurrent in (False, True):
        a, b = run_fwd(q, k, v, d, None, None, recurrent=recurrent), run_fwd(*c, d, None, None, recurrent=recurrent)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = linattn.bwd(q, k, v, d, SCALE, do), linattn.bwd(*c, d, SCALE, do)
    assert all(torch.equal(a[m], b[m]) for m in ("dq", "dk", "dv", "ddecay", "dinitial_state"))


def test_state_past_32_bits():
    """Decode on states of more than 2^31 elements, in place: the first and the last sequences."""
    N, H = 4100, 32
    q, k, v, d, n = inputs(N, 1, 2, H, 82)
    h = torch.zeros(N, H, D, D, dtype=torch.bfloat16, device=dev())
    assert h.numel() > 2 ** 31
    ends = torch.tensor([0, 1, N // 2, N - 1], device=dev())
    h[ends] = states(4, H, torch.bfloat16, n)
    ro, rs = lin_ref(q[ends], k[ends], v[ends], d[ends], SCALE, h[ends])
    h1 = h[ends].clone()
    out, _ = run_fwd(q, k, v, d, h, None, recurrent=True, in_place=True)
    close_bf16(out[ends], ro, "out")
    close_bf16(h[ends], rs, "final")
    h[ends] = h1
    out, _ = run_fwd(q, k, v, d, h, None, in_place=True)
    close_bf16(out[ends], ro, "out")
    close_bf16(h[ends], rs, "final")
