"""The gated delta rule and the norms around it run together as a layer uses them: projections -> q/k norm and rotation ->
gated delta rule -> gated norm -> residual step; a prompt, then decode steps on the carried state; a training step through
all backward passes; captured graphs, other streams and used workspaces."""
import pytest
import torch

from gated_delta_rule_86_amd import blocknorm, gdn, qkrope

from gdn_testutil import (BF16_STEP, D, FP32_MAX, FP32_REL_L2, close_bf16, close_fp32, close_grads, gdn_ref, gdn_ref_bwd,
                          inputs)
from test_gpu_blocknorm import act, rms
from test_gpu_qkrope import ref as rope_ref

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


def layer_inputs(B, T, Hk, H, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    wide = n(B, T, (2 * Hk + 2 * H) * D).bfloat16()
    q, k, v, z = (x.unflatten(2, (-1, D)) for x in wide.split([Hk * D, Hk * D, H * D, H * D], -1))
    decay = -(1e-3 ** torch.rand((B, T, H), generator=g, device="cuda"))
    beta = torch.rand((B, T, H), generator=g, device="cuda")
    f, m = qkrope.inv_freq(D // 2, device="cuda")
    return dict(q=q, k=k, v=v, z=z, decay=decay, beta=beta, stream=n(B, T, H * D).bfloat16(), f=f, m=m,
                w=1 + 0.1 * n(D), wn=1 + 0.1 * n(H * D), scale=0.5 + 0.1 * n(H * D)), n


def buffers(s):
    B, T, Hk, _ = s["q"].shape
    H = s["v"].shape[2]
    e = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    return e(B, T, Hk, D), e(B, T, Hk, D), e(B, T, H, D), e(B, T, H, D), e(B, T, H * D), e(B, T, H * D)


def layer(s, pos, bufs, h0, ht, step=gdn.fwd, **kw):
    """The layer's forward pass into bufs: q', k', o, y, out, residual_out."""
    a, b, o, y, out, res = bufs
    qkrope.fwd(s["q"], s["k"], pos, s["f"], a, b, norm="l2", attention_factor=s["m"])
    step(a, b, s["v"], s["decay"], s["beta"], SCALE, o, h0, ht, **kw)
    blocknorm.gated(o, s["z"], y, weight=s["w"], activation="silu")
    blocknorm.residual(y.flatten(2), s["stream"], out, res, weight=s["wn"], scale=s["scale"])
    return bufs


def layer_bwd(s, pos, bufs, h0, dout, dres, dht, **kw):
    a, b, o, y, out, res = bufs
    r = blocknorm.residual_bwd(y.flatten(2), res, dout, dres, weight=s["wn"], scale=s["scale"])
    g = blocknorm.gated_bwd(o, s["z"], r["dx"].view(o.shape), weight=s["w"], activation="silu")
    d = gdn.bwd(a, b, s["v"], s["decay"], s["beta"], SCALE, g["dx"], h0, dht, **kw)
    p = qkrope.bwd(s["q"], s["k"], pos, s["f"], d["dq"], d["dk"], norm="l2", attention_factor=s["m"])
    return dict(dq=p["dq"], dk=p["dk"], dv=d["dv"], dz=g["dgate"], ddecay=d["ddecay"], dbeta=d["dbeta"],
                dstream=r["dresidual"], dw=g["dweight"], dwn=r["dweight"], dscale=r["dscale"], dh0=d["dinitial_state"])


@pytest.mark.parametrize("T,steps", [(1, 1), (63, 2), (200, 3), (1500, 2)])
def test_prompt_then_decode(T, steps):
    """A prompt and `steps` single tokens, the state carried in place, equal one run of T + steps tokens: the delta rule against
    64 bits from the q', k' it read, each norm from the values it read."""
    B, Hk, H = 2, 2, 4
    s, n = layer_inputs(B, T + steps, Hk, H, T)
    pos = (100000 + torch.arange(T + steps, device="cuda")).repeat(B, 1)
    state = (0.5 * n(B, H, D, D)).contiguous()
    h0, parts = state.clone(), []
    for lo, hi in [(0, T)] + [(T + i, T + i + 1) for i in range(steps)]:
        part = {name: x[:, lo:hi] if name in ("q", "k", "v", "z", "stream") else
                x[:, lo:hi].contiguous() if name in ("decay", "beta") else x for name, x in s.items()}
        parts.append(layer(part, pos[:, lo:hi].contiguous(), buffers(part), state, state,
                           gdn.fwd if lo == 0 else gdn.fwd_recurrent))
    a, b, o, y, out, res = (torch.cat(x, 1) for x in zip(*parts))
    ro, rs = gdn_ref(a, b, s["v"], s["decay"], s["beta"], SCALE, h0)
    close_bf16(o, ro, "o")
    close_fp32(state, rs, "state")
    close_bf16(y, rms(o.double(), s["w"].double(), 1e-6) * act(s["z"].double(), "silu"), "y")
    stream = s["stream"].double() + s["scale"].double() * y.flatten(2).double()
    close_bf16(res, stream, "residual_out")
    close_bf16(out, rms(stream, s["wn"].double(), 1e-6), "out")


def test_training_step():
    """Gradients through the four backward passes against automatic differentiation of the whole layer in fp64.  Along a path lie
    at most nine roundings to bf16 of 2^-8 each (q' and k', o, y, residual_out; then dy, do, dq' or dk', and the gradient
    itself): 9 * 2^-8 in the norm."""
    B, T, Hk, H = 2, 150, 2, 4
    s, n = layer_inputs(B, T, Hk, H, 7)
    pos = torch.arange(T, device="cuda").repeat(B, 1)
    h0, dht = 0.5 * n(B, H, D, D), n(B, H, D, D)
    ht = torch.empty_like(h0)
    dout, dres = n(B, T, H * D).bfloat16(), n(B, T, H * D).bfloat16()
    bufs = layer(s, pos, buffers(s), h0, ht)
    got = layer_bwd(s, pos, bufs, h0, dout, dres, dht)

    names = dict(dq="q", dk="k", dv="v", dz="z", ddecay="decay", dbeta="beta", dstream="stream", dw="w", dwn="wn",
                 dscale="scale")
    leaf = {x: s[x].double().contiguous().requires_grad_() for x in names.values()}
    start = h0.double().requires_grad_()
    rope = lambda x: rope_ref(x, None, pos, s["f"], "l2", 1e-6, False, s["m"])  # noqa: E731
    o, final = gdn_ref(rope(leaf["q"]), rope(leaf["k"]), leaf["v"], leaf["decay"], leaf["beta"], SCALE, start)
    y = rms(o, leaf["w"], 1e-6) * act(leaf["z"], "silu")
    res = leaf["stream"] + leaf["scale"] * y.flatten(2)
    out = rms(res, leaf["wn"], 1e-6)
    loss = (out * dout.double()).sum() + (res * dres.double()).sum() + (final * dht.double()).sum()
    want = torch.autograd.grad(loss, list(leaf.values()) + [start])
    for name, x in zip(list(names) + ["dh0"], want):
        rel = float((got[name].double() - x).norm() / x.norm())
        assert rel <= 9 * BF16_STEP, (name, rel)


@pytest.mark.parametrize("cu", [None, [0, 100, 100, 101, 1300]], ids=["rows", "packed"])
def test_captured_and_replayed(cu):
    """A training step in a graph, its workspaces outside of it, replayed with other inputs and eager work in between: the
    bits of the eager calls."""
    B, T, Hk, H = (2, 1100, 2, 4) if cu is None else (1, 1300, 2, 4)
    s, n = layer_inputs(B, T, Hk, H, 11)
    N = B if cu is None else len(cu) - 1
    c = None if cu is None else torch.tensor(cu, dtype=torch.int64, device="cuda")
    pos = torch.arange(T, device="cuda").repeat(B, 1)
    h0, dht = 0.5 * n(N, H, D, D), n(N, H, D, D)
    ht = torch.empty_like(h0)
    dout, dres = n(B, T, H * D).bfloat16(), n(B, T, H * D).bfloat16()
    bufs = buffers(s)
    wf = torch.empty(gdn.workspace_size(B, T, H, N, c is not None), dtype=torch.uint8, device="cuda")
    wb = torch.empty(gdn.bwd_workspace_size(B, T, Hk, H, N, c is not None), dtype=torch.uint8, device="cuda")

    def step():
        layer(s, pos, bufs, h0, ht, cu_seqlens=c, workspace=wf)
        return layer_bwd(s, pos, bufs, h0, dout, dres, dht, cu_seqlens=c, workspace=wb)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        s["q"].copy_(n(*s["q"].shape))
        s["v"].copy_(n(*s["v"].shape))
        s["decay"].copy_(-torch.rand_like(s["decay"]))
        dout.copy_(n(*dout.shape))
        graph.replay()
        torch.cuda.synchronize()
        replayed = [x.clone() for x in (*bufs, ht, *got.values())]
        want = step()
        torch.cuda.synchronize()
        for x, y in zip(replayed, (*bufs, ht, *want.values())):
            assert torch.equal(x, y), i


def test_two_calls_at_once():
    """Forward and backward passes on two streams at the same time, each with its own workspace, against one after the other."""
    cases = [inputs(2, 1500, 2, 4, 1), inputs(1, 2100, 1, 3, 2)]
    douts = [a[-1](*a[2].shape).bfloat16() for a in cases]

    def run(i, stream):
        q, k, v, decay, beta, _ = cases[i]
        out, ht = torch.empty_like(v), torch.empty(v.shape[0], v.shape[2], D, D, device="cuda")
        gdn.fwd(q, k, v, decay, beta, SCALE, out, None, ht, stream=stream)
        r = gdn.bwd(q, k, v, decay, beta, SCALE, douts[i], stream=stream)
        return [out, ht, *(x for name, x in r.items() if name != "workspace")]

    want = []
    for i in range(2):
        want.append(run(i, None))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for t in streams:
        t.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = [run(i, streams[i]) for i in range(2)]
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(x, y))


@pytest.mark.parametrize("lens", [[700, 0, 1, 333], [1500], [33, 64, 65, 31, 1, 0, 90]], ids=str)
def test_used_workspace(lens):
    """What a workspace holds before a call, NaN among it, changes nothing."""
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int64, device="cuda")
    T, N = sum(lens), len(lens)
    q, k, v, decay, beta, n = inputs(1, T, 1, 2, T)
    h0, dht, dout = n(N, 2, D, D), n(N, 2, D, D), n(1, T, 2, D).bfloat16()
    got = []
    for fill in (0, 255):
        wf = torch.full((gdn.workspace_size(1, T, 2, N, True),), fill, dtype=torch.uint8, device="cuda")
        wb = torch.full((gdn.bwd_workspace_size(1, T, 1, 2, N, True),), fill, dtype=torch.uint8, device="cuda")
        out, ht = torch.empty_like(v), torch.empty_like(h0)
        gdn.fwd(q, k, v, decay, beta, SCALE, out, h0, ht, cu, workspace=wf)
        r = gdn.bwd(q, k, v, decay, beta, SCALE, dout, h0, dht, cu, workspace=wb)
        got.append([out, ht, *(r[x] for x in ("dq", "dk", "dv", "ddecay", "dbeta", "dinitial_state"))])
    torch.cuda.synchronize()
    for x, y in zip(*got):
        assert torch.isfinite(x).all() and torch.equal(x, y)


def test_many_short_sequences():
    """2000 sequences of 0 to 5 tokens; each equals its own call of one row."""
    N, H = 2000, 2
    lens = [(7 * i) % 6 for i in range(N)]
    cu = [0]
    for m in lens:
        cu.append(cu[-1] + m)
    q, k, v, decay, beta, n = inputs(1, cu[-1], 1, H, 3)
    h0, dht, dout = n(N, H, D, D), n(N, H, D, D), n(1, cu[-1], H, D).bfloat16()
    c = torch.tensor(cu, dtype=torch.int64, device="cuda")
    out, ht = torch.empty_like(v), torch.empty_like(h0)
    gdn.fwd(q, k, v, decay, beta, SCALE, out, h0, ht, c)
    r = gdn.bwd(q, k, v, decay, beta, SCALE, dout, h0, dht, c)
    for i in [0, 1, 2, 5, 777, 1996, 1999]:
        t = slice(cu[i], cu[i + 1])
        part = [x[:, t] for x in (q, k, v)] + [x[:, t].contiguous() for x in (decay, beta)]
        o, f = torch.empty(1, lens[i], H, D, dtype=torch.bfloat16, device="cuda"), torch.empty_like(ht[i:i + 1])
        gdn.fwd(*part, SCALE, o, h0[i:i + 1], f)
        p = gdn.bwd(*part, SCALE, dout[:, t].contiguous(), h0[i:i + 1], dht[i:i + 1])
        assert torch.equal(o, out[:, t]) and torch.equal(f, ht[i:i + 1]), i
        for name in ("dq", "dk", "dv", "ddecay", "dbeta"):
            assert torch.equal(p[name], r[name][:, t]), (i, name)
        assert torch.equal(p["dinitial_state"], r["dinitial_state"][i:i + 1]), i


def test_broadcast_batch():
    """q, k and v of one row for a whole batch (stride 0), states of their own."""
    q, k, v, decay, beta, n = inputs(1, 90, 2, 2, 9)
    q, k, v = (x.expand(3, -1, -1, -1) for x in (q, k, v))
    decay, beta = decay.repeat(3, 1, 1), beta.repeat(3, 1, 1)
    h0, dout = n(3, 2, D, D), n(3, 90, 2, D).bfloat16()
    got = []
    for f in (lambda x: x, lambda x: x.contiguous()):
        out, ht = torch.empty(3, 90, 2, D, dtype=torch.bfloat16, device="cuda"), torch.empty_like(h0)
        gdn.fwd(f(q), f(k), f(v), decay, beta, SCALE, out, h0, ht)
        r = gdn.bwd(f(q), f(k), f(v), decay, beta, SCALE, dout, h0)
        one, st = torch.empty_like(out[:, :1]), torch.empty_like(h0)
        gdn.fwd_recurrent(f(q)[:, :1], f(k)[:, :1], f(v)[:, :1], decay[:, :1].contiguous(), beta[:, :1].contiguous(), SCALE, one,
                          h0, st)
        got.append([out, ht, one, st, *(x for name, x in r.items() if name != "workspace")])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*got))


@pytest.mark.parametrize("packed", [False, True])
def test_offsets_past_32_bits(packed):
    """v, out and their gradients of more than 2^31 elements: decays of -1 leave 2^-369 of what lies 256 tokens back, so the last
    tokens are those of a short call over the end."""
    T, H, tail, keep = (1 << 20) + 77, 17, 1000, 500
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    q, k = (torch.nn.functional.normalize(torch.randn((1, T, 1, D), generator=g, device="cuda"), dim=-1).bfloat16()
            for _ in range(2))
    v = torch.empty(1, T, H, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    assert v.numel() > 1 << 31
    decay, beta = torch.full((1, T, H), -1.0, device="cuda"), torch.rand((1, T, H), generator=g, device="cuda")
    dout = torch.empty_like(v).normal_(generator=g)
    c = torch.tensor([0, T], dtype=torch.int64, device="cuda") if packed else None
    out, ht = torch.empty_like(v), torch.empty(1, H, D, D, device="cuda")
    gdn.fwd(q, k, v, decay, beta, SCALE, out, None, ht, c)
    r = gdn.bwd(q, k, v, decay, beta, SCALE, dout, None, None, c, need_dinitial_state=False)
    last = lambda x, m: x[:, -m:].contiguous()  # noqa: E731
    o, f = torch.empty(1, tail, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty_like(ht)
    part = [last(x, tail) for x in (q, k, v, decay, beta)]
    gdn.fwd(*part, SCALE, o, None, f)
    p = gdn.bwd(*part, SCALE, last(dout, tail), need_dinitial_state=False)
    # the same formulas in other chunks: two results that are each as close to the exact one as the tests of that allow, so
    # two half steps apart and twice the fp32 sums' share
    close_fp32(ht, f, "state", 2 * FP32_REL_L2, 2 * FP32_MAX)
    r["out"], p["out"] = out, o
    for name in ("out", "dq", "dk", "dv"):
        a, b = last(r[name], keep).double(), last(p[name], keep).double()
        rms_b = b.square().mean().sqrt()
        assert ((a - b).abs() <= 2 * BF16_STEP * torch.maximum(a.abs(), b.abs()) + 2.0 ** -15 * rms_b).all(), name
    for name in ("ddecay", "dbeta"):
        a, b = last(r[name], keep).double(), last(p[name], keep).double()
        assert float((a - b).norm()) <= 2 * 8 * FP32_REL_L2 * float(b.norm()) * D ** 0.5, name


def test_state_past_32_bits():
    """A decode step over a state of more than 2^31 elements, in place; the last sequences against a call of their own."""
    N, H = 4100, 32
    q, k, v, decay, beta, n = inputs(N, 1, 1, H, 21)
    state = torch.empty(N, H, D, D, device="cuda").normal_()
    assert state.numel() > 1 << 31
    part = [x[-3:].contiguous() for x in (q, k, v, decay, beta)]
    st = state[-3:].clone()
    out, o = torch.empty_like(v), torch.empty_like(part[2])
    gdn.fwd_recurrent(*part, SCALE, o, st, st)
    gdn.fwd_recurrent(q, k, v, decay, beta, SCALE, out, state, state)
    torch.cuda.synchronize()
    assert torch.equal(out[-3:], o) and torch.equal(state[-3:], st)


@pytest.mark.parametrize("cu", [None, [0, 1, 3100, 3100, 7500]], ids=["rows", "packed"])
def test_long_segments_of_many_heads(cu):
    """70 heads in segments of more than 1000 tokens, where heads that forget slowly are taken first, among the first 64 and
    behind them: some heads of either kind against the reference."""
    T, H, some = 7500, 70, [0, 31, 63, 66, 69]
    N = 1 if cu is None else len(cu) - 1
    q, k, v, decay, beta, n = inputs(1, T, H, H, 41)
    decay = decay * torch.where(torch.arange(H, device="cuda") % 3 == 0, 1e-2, 1.0)
    h0, dht, dout = n(N, H, D, D), n(N, H, D, D), n(1, T, H, D).bfloat16()
    c = None if cu is None else torch.tensor(cu, dtype=torch.int64, device="cuda")
    out, ht = torch.empty_like(v), torch.empty_like(h0)
    gdn.fwd(q, k, v, decay, beta, SCALE, out, h0, ht, c)
    r = gdn.bwd(q, k, v, decay, beta, SCALE, dout, h0, dht, c)
    args = [x[:, :, some].contiguous() for x in (q, k, v, decay, beta)]
    ro, rs = gdn_ref(*args, SCALE, h0[:, some], cu)
    close_bf16(out[:, :, some], ro, "out")
    close_fp32(ht[:, some], rs, "final")
    want = gdn_ref_bwd(*args, SCALE, dout[:, :, some], h0[:, some], dht[:, some], cu)
    got = {x: r[x][:, :, some] for x in ("dq", "dk", "dv", "ddecay", "dbeta")}
    close_grads(got | {"dinitial_state": r["dinitial_state"][:, some]}, want)
