"""Refusals and sizes of kda_gdn_*, kda_gated_norm* and kda_residual_norm* (no GPU: every check runs before any HIP call, the fake
pointers are never dereferenced), and the 64-bit reference of the gated delta rule against automatic differentiation and
against differences."""
import ctypes

import numpy as np
import pytest
import torch

from gated_delta_rule_86_amd import blocknorm, gdn, kda

from gdn_testutil import D, gdn_ref, gdn_ref_bwd, inputs

STEP = 1 << 42
BASE = 1 << 46


def ptr(i):
    return BASE + i * STEP


def gdn_args(**ch):
    a = dict(q=ptr(0), k=ptr(1), v=ptr(2), decay=ptr(3), beta=ptr(16), scale=0.1, out=ptr(4), h0=ptr(5), h0_dt=2,
             ht=ptr(6), ht_dt=2, cu=None, cu_host=None, B=2, T=100, Hk=2, H=4, N=0, K=128, V=128, strides=None,
             ws=ptr(7), ws_bytes=1 << 31, dout=ptr(9), dht=ptr(10), dq=ptr(11), dk=ptr(12), dv=ptr(13), dd=ptr(14),
             db=ptr(17), dh0=ptr(15))
    a.update(ch)
    if a["strides"] is not None:
        a["strides"] = (ctypes.c_int64 * len(a["strides"]))(*a["strides"])
    if a["cu_host"] is not None:
        a["cu_host"] = np.array(a["cu_host"], dtype=np.int64)
    return a


def gdn_call(name, **ch):
    a = gdn_args(**ch)
    host = None if a["cu_host"] is None else a["cu_host"].ctypes.data
    first = (a["q"], a["k"], a["v"], a["decay"], a["beta"], a["scale"])
    last = (a["cu"], host, a["B"], a["T"], a["Hk"], a["H"], a["N"], a["K"], a["V"], a["strides"], a["ws"], a["ws_bytes"], None)
    if name == "kda_gdn_bwd":
        return kda.lib().kda_gdn_bwd(*first, a["h0"], a["h0_dt"], a["dout"], a["dht"], a["dq"], a["dk"], a["dv"], a["dd"],
                                     a["db"], a["dh0"], *last)
    return getattr(kda.lib(), name)(*first, a["out"], a["h0"], a["h0_dt"], a["ht"], a["ht_dt"], *last)


BOTH = [
    (1, dict(q=None)), (1, dict(k=None)), (1, dict(v=None)), (1, dict(decay=None)), (1, dict(beta=None)),
    (2, dict(B=0)), (2, dict(T=-1)), (2, dict(H=0, Hk=1)), (2, dict(N=3)), (2, dict(cu=ptr(8), N=2)),
    (2, dict(B=1, cu=ptr(8), N=0)), (2, dict(T=1 << 36)), (2, dict(B=1 << 29, T=1, H=64)),
    (2, dict(B=1, cu=ptr(8), N=1 << 28, H=4)), (2, dict(T=1 << 34, H=1 << 16, Hk=1)),
    (3, dict(K=64)), (3, dict(V=256)), (4, dict(h0_dt=0)), (4, dict(h0_dt=3)), (4, dict(h0=None)),
    (6, dict(scale=float("nan"))), (6, dict(scale=float("inf"))),
    (7, dict(q=ptr(0) + 8)), (7, dict(decay=ptr(3) + 2)), (7, dict(beta=ptr(16) + 1)), (7, dict(ws=ptr(7) + 128)),
    (7, dict(h0=ptr(5) + 8)), (7, dict(B=1, cu=ptr(8) + 4, N=2)),
    (14, dict(H=3)), (14, dict(Hk=0)), (14, dict(Hk=8)),
    (15, dict(strides=[8, 4, 128] * 3)), (15, dict(strides=[0, -8, 128] * 3)), (15, dict(strides=[0, 1 << 25, 128] * 3)),
    (15, dict(strides=[0, 256, 128, 0, 256, 128, 0, 512, 100])), (15, dict(strides=[0, 0, 0] * 3)),
    (15, dict(strides=[0, 120, 128] * 3)),
    (9, dict(B=1, cu=ptr(8), N=2, cu_host=[0, 50, 99])), (9, dict(B=1, cu=ptr(8), N=2, cu_host=[1, 50, 100])),
    (9, dict(B=1, cu=ptr(8), N=2, cu_host=[0, 101, 100])), (8, dict(B=1, cu=ptr(8), N=2, ws=None)),
    (8, dict(B=1, cu=ptr(8), N=2, ws_bytes=255)), (11, dict(ws=ptr(2))), (11, dict(ws=ptr(16))),
]


@pytest.mark.parametrize("code,change", BOTH, ids=str)
@pytest.mark.parametrize("name", ["kda_gdn_fwd", "kda_gdn_fwd_recurrent", "kda_gdn_bwd"])
def test_refusals(name, code, change):
    assert gdn_call(name, **change) == code


@pytest.mark.parametrize("code,change", [
    (1, dict(out=None)), (4, dict(ht_dt=0)), (4, dict(ht_dt=1)), (4, dict(h0_dt=1)), (7, dict(out=ptr(4) + 2)), (11, dict(out=ptr(0))),
    (11, dict(out=ptr(2))), (11, dict(ht=ptr(1))), (11, dict(ht=ptr(5) + 4096)), (11, dict(out=ptr(5))),
    (11, dict(out=ptr(3))), (11, dict(out=ptr(16))), (11, dict(ht=ptr(4))),
], ids=str)
@pytest.mark.parametrize("name", ["kda_gdn_fwd", "kda_gdn_fwd_recurrent"])
def test_forward_refusals(name, code, change):
    assert gdn_call(name, **change) == code


@pytest.mark.parametrize("code,change", [
    (1, dict(dout=None)), (1, dict(dq=None)), (1, dict(dk=None)), (1, dict(dv=None)), (1, dict(dd=None)), (1, dict(db=None)),
    (7, dict(dout=ptr(9) + 8)), (7, dict(dk=ptr(12) + 8)), (7, dict(dd=ptr(14) + 1)), (7, dict(dh0=ptr(15) + 4)),
    (11, dict(dq=ptr(0))), (11, dict(dq=ptr(9))), (11, dict(dk=ptr(11))), (11, dict(dh0=ptr(10))), (11, dict(dd=ptr(3))),
    (11, dict(db=ptr(16))), (11, dict(db=ptr(14))), (11, dict(dh0=ptr(5))), (11, dict(ws=ptr(13))),
    (8, dict(ws=None)), (8, dict(ws_bytes=1024)),
], ids=str)
def test_backward_refusals(code, change):
    assert gdn_call("kda_gdn_bwd", **change) == code


def test_workspaces():
    need = gdn.workspace_size(2, 100, 4)
    assert gdn_call("kda_gdn_fwd", ws_bytes=need - 1) == 8
    assert gdn.workspace_size(3, 0, 2) == 256 and gdn.workspace_size(0, 10, 1) == 0
    assert gdn.workspace_size(2, 10, 1, 3, True) == 0 and gdn.bwd_workspace_size(1, 64, 2, 3) == 0
    shared, alone = gdn.bwd_workspace_size(4, 100, 2, 4), gdn.bwd_workspace_size(4, 100, 4, 4)
    assert shared - alone == 2 * 4 * 100 * 4 * 512
    # a chunk's place is floor(begin / 32) + sequence + chunk, a block's the same with 64: enough for any lengths
    rng = np.random.default_rng(1)
    for n in range(400):
        lens, C = rng.integers(0, 200, rng.integers(1, 20)), 32 << (n & 1)
        begin = np.concatenate([[0], lens.cumsum()])
        seen = [begin[i] // C + i + c for i in range(len(lens)) for c in range(-(-lens[i] // C))]
        assert len(set(seen)) == len(seen) and (not seen or max(seen) < begin[-1] // C + len(lens) + 1)


@pytest.mark.parametrize("name", ["kda_gdn_fwd", "kda_gdn_bwd"])
def test_launch_limits(name):
    """Sizes whose launch would hold 2^32 threads or more are refused by the checks, not by the runtime."""
    small = dict(h0=None, h0_dt=0, ht=None, ht_dt=0, ws=None, dht=None, dh0=None)
    most = (1 << 26) // 4 * 32 if name == "kda_gdn_fwd" else (1 << 23) // 4 * 64   # chunks, blocks times heads
    assert gdn_call(name, B=1, T=most - 1024, H=4, Hk=1, **small) == 8
    assert gdn_call(name, B=1, T=most, H=4, Hk=1, **small) == 2
    assert gdn_call("kda_gdn_fwd_recurrent", B=1, cu=ptr(8), N=1 << 22, **small) == 2
    assert gdn_call("kda_gdn_fwd_recurrent", B=1, cu=ptr(8), N=(1 << 22) - 2, **small) == 8


def gated_call(back=False, **ch):
    a = dict(x=ptr(0), z=ptr(1), w=ptr(2), y=ptr(3), dy=ptr(4), dz=ptr(5), dw=ptr(6), B=2, T=10, H=4, D=128, dtype=1, act=0,
             eps=1e-6, strides=None, ws=ptr(7), ws_bytes=1 << 24)
    a.update(ch)
    st = None if a["strides"] is None else (ctypes.c_int64 * len(a["strides"]))(*a["strides"])
    sizes = (a["B"], a["T"], a["H"], a["D"], a["dtype"], a["act"], a["eps"], st)
    if back:
        return kda.lib().kda_gated_norm_bwd(a["x"], a["z"], a["w"], a["dy"], a["y"], a["dz"], a["dw"], *sizes, a["ws"],
                                            a["ws_bytes"], None)
    return kda.lib().kda_gated_norm(a["x"], a["z"], a["w"], a["y"], *sizes, None)


@pytest.mark.parametrize("code,change", [
    (1, dict(x=None)), (1, dict(z=None)), (1, dict(y=None)), (2, dict(B=0)), (2, dict(T=-1)), (2, dict(H=0)),
    (2, dict(T=1 << 31)), (2, dict(B=1 << 15, T=1 << 14)), (2, dict(H=1 << 17)), (3, dict(D=0)), (3, dict(D=12)), (3, dict(D=520)),
    (4, dict(dtype=0)), (4, dict(dtype=4)), (12, dict(act=2)), (12, dict(act=-1)), (6, dict(eps=-1.0)), (6, dict(eps=float("nan"))),
    (6, dict(eps=float("inf"))), (7, dict(x=ptr(0) + 8)), (7, dict(y=ptr(3) + 2)), (7, dict(w=ptr(2) + 2)),
    (11, dict(y=ptr(0) + 16)), (11, dict(y=ptr(2))), (15, dict(strides=[0, 4, 128, 0, 512, 128])),
    (15, dict(strides=[-8, 512, 128] * 2)), (15, dict(strides=[0, 512, 128, 0, 1 << 47, 128])),
    (15, dict(dtype=2, strides=[0, 512, 130, 0, 512, 128])),
    (11, dict(y=ptr(0), strides=[5120, 1024, 128, 5120, 512, 128])),   # in place on a view
], ids=str)
@pytest.mark.parametrize("back", [False, True])
def test_gated_refusals(back, code, change):
    assert gated_call(back, **change) == code


@pytest.mark.parametrize("code,change", [
    (1, dict(dy=None)), (1, dict(dz=None)), (1, dict(w=None)), (11, dict(y=ptr(0))), (11, dict(y=ptr(4))), (11, dict(dz=ptr(3))),
    (11, dict(dw=ptr(2))), (11, dict(ws=ptr(1))), (7, dict(dw=ptr(6) + 1)), (7, dict(ws=ptr(7) + 16)), (8, dict(ws=None)),
    (8, dict(ws_bytes=100)),
], ids=str)
def test_gated_backward_refusals(code, change):
    assert gated_call(True, **change) == code


def residual_call(back=False, **ch):
    a = dict(x=ptr(0), z=ptr(1), w=ptr(2), sc=ptr(3), pw=ptr(4), y=ptr(5), zo=ptr(6), dy=ptr(7), dzo=ptr(8), dw=ptr(9),
             dsc=ptr(10), dpw=ptr(11), B=2, T=10, D=128, dtype=1, rdtype=2, post=1, eps=1e-6, strides=None, ws=ptr(12),
             ws_bytes=1 << 24)
    a.update(ch)
    st = None if a["strides"] is None else (ctypes.c_int64 * len(a["strides"]))(*a["strides"])
    sizes = (a["B"], a["T"], a["D"], a["dtype"], a["rdtype"], a["post"], a["eps"], st)
    if back:
        return kda.lib().kda_residual_norm_bwd(a["x"], a["z"], a["dy"], a["dzo"], a["w"], a["sc"], a["pw"], a["y"], a["zo"],
                                               a["dw"], a["dsc"], a["dpw"], *sizes, a["ws"], a["ws_bytes"], None)
    return kda.lib().kda_residual_norm(a["x"], a["z"], a["w"], a["sc"], a["pw"], a["y"], a["zo"], *sizes, None)


@pytest.mark.parametrize("code,change", [
    (1, dict(x=None)), (1, dict(z=None)), (1, dict(y=None)), (1, dict(zo=None)), (2, dict(B=0)), (2, dict(T=-1)),
    (2, dict(T=1 << 31)), (3, dict(D=4)), (3, dict(D=100)), (3, dict(D=8200)), (4, dict(dtype=0)), (4, dict(rdtype=3)),
    (4, dict(dtype=2, rdtype=1)), (12, dict(post=2)), (12, dict(post=0)), (6, dict(eps=-1.0)), (6, dict(eps=float("nan"))),
    (7, dict(z=ptr(1) + 8)), (7, dict(zo=ptr(6) + 4)), (7, dict(sc=ptr(3) + 2)), (11, dict(y=ptr(1))), (11, dict(zo=ptr(0))),
    (11, dict(y=ptr(6))), (11, dict(zo=ptr(4))), (11, dict(y=ptr(0) + 16)), (15, dict(strides=[0, 132, 0, 128])),
    (15, dict(strides=[0, -128, 0, 128])), (11, dict(y=ptr(0), strides=[2560, 256, 1280, 128])),
], ids=str)
@pytest.mark.parametrize("back", [False, True])
def test_residual_refusals(back, code, change):
    assert residual_call(back, **change) == code


@pytest.mark.parametrize("code,change", [
    (1, dict(dy=None)), (1, dict(w=None)), (1, dict(sc=None)), (1, dict(pw=None)), (11, dict(y=ptr(0))), (11, dict(zo=ptr(1))),
    (11, dict(zo=ptr(8))), (11, dict(dw=ptr(10))), (11, dict(ws=ptr(7))), (7, dict(dpw=ptr(11) + 2)), (7, dict(ws=ptr(12) + 8)),
    (8, dict(ws=None)), (8, dict(ws_bytes=1000)),
], ids=str)
def test_residual_backward_refusals(code, change):
    assert residual_call(True, **change) == code


def test_python_refusals():
    """What the bindings refuse before the library is called."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    f32 = torch.float32
    q, v, d, out = z(1, 4, 2, 128), z(1, 4, 4, 128), z(1, 4, 4, dt=f32), z(1, 4, 4, 128)
    for bad in (dict(q=z(1, 4, 256)), dict(q=q.float()), dict(k=z(1, 5, 2, 128)), dict(v=z(1, 5, 4, 128)), dict(d=z(4, dt=f32)),
                dict(d=z(1, 4, 3, dt=f32)), dict(d=z(1, 4, 4)), dict(b=z(1, 4, 4)), dict(b=z(1, 4, 3, dt=f32)), dict(b=z(4, dt=f32)),
                dict(b=z(1, 4, 4, dt=f32).mT), dict(out=z(1, 4, 4, 64)), dict(out=out.float())):
        a = dict(q=q, k=q, v=v, d=d, b=d, out=out) | bad
        with pytest.raises(ValueError):
            gdn.fwd(a["q"], a["k"], a["v"], a["d"], a["b"], 1.0, a["out"])
    s = z(1, 4, 128, 128, dt=f32)
    for kw in (dict(initial_state=s[:, :2]), dict(initial_state=s.half()), dict(initial_state=s, final_state=s.bfloat16()),
               dict(final_state=s.mT), dict(cu_seqlens=torch.zeros(2, dtype=torch.int32)), dict(cu_seqlens_host=[0, 4])):
        with pytest.raises(ValueError):
            gdn.fwd(q, q, v, d, d, 1.0, out, **kw)
    for kw in (dict(dout=out.float()), dict(dout=out[:, :2]), dict(dfinal_state=s.bfloat16())):
        with pytest.raises(ValueError):
            gdn.bwd(q, q, v, d, d, 1.0, **(dict(dout=out) | kw))
    x, w = z(2, 3, 2, 64), z(64, dt=f32)
    for a, kw in (((x, x.float(), x), {}), ((x, x[:, :2], x), {}), ((x, x, x.float()), {}), ((x, x, x.mT), {}),
                  ((x.double(),) * 3, {}), ((x[0],) * 3, {}), ((x, x, x), dict(weight=w.half())), ((x, x, x), dict(weight=w[:32])),
                  ((x, x, x), dict(activation="tanh"))):
        with pytest.raises(ValueError):
            blocknorm.gated(*a, **kw)
        with pytest.raises(ValueError):
            blocknorm.gated_bwd(*a, **kw)
    x = z(2, 3, 64)
    for a, kw in (((x, x.half(), x, x), {}), ((x, x[:, :2], x, x), {}), ((x, x, x.float(), x), {}), ((x, x, x, x.float()), {}),
                  ((x.double(),) * 4, {}), ((x[0],) * 4, {}), ((x, x, x, x), dict(scale=w.half())),
                  ((x, x, x, x), dict(post_norm="l2")), ((x, x, x, x), dict(weight=z(32, dt=f32)))):
        with pytest.raises(ValueError):
            blocknorm.residual(*a, **kw)
        with pytest.raises(ValueError):
            blocknorm.residual_bwd(*a, **kw)


@pytest.mark.parametrize("Hk,H,cu", [(1, 2, None), (2, 2, [0, 3, 3, 7])])
def test_reference_gradients(Hk, H, cu):
    """The recurrence run backwards against automatic differentiation, and that against differences along random directions."""
    q, k, v, d, b, n = inputs(1, 7, Hk, H, 3, lo=1e-2, device="cpu")
    N = 1 if cu is None else len(cu) - 1
    h0, dht, dout = n(N, H, D, D), n(N, H, D, D), n(*v.shape).bfloat16()
    leaves = [x.double().requires_grad_() for x in (q, k, v, d, b, h0)]

    def loss(q, k, v, d, b, h0):
        out, fin = gdn_ref(q, k, v, d, b, 0.3, h0, cu)
        return (out * dout.double()).sum() + (fin * dht.double()).sum()
    grads = torch.autograd.grad(loss(*leaves), leaves)
    want = gdn_ref_bwd(q, k, v, d, b, 0.3, dout, h0, dht, cu)
    for x, name in zip(grads, ("dq", "dk", "dv", "ddecay", "dbeta", "dinitial_state")):
        assert torch.allclose(want[name], x, rtol=1e-10, atol=1e-10 * float(x.abs().max()))
    with torch.no_grad():
        for i, g in enumerate(grads):
            u = torch.randn(g.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(i))
            e = 1e-6
            plus, minus = ([x + s * e * u if j == i else x for j, x in enumerate(leaves)] for s in (1, -1))
            got = (loss(*plus) - loss(*minus)) / (2 * e)
            assert abs(got - (g * u).sum()) <= 1e-6 * float(g.norm() * u.norm())
