"""Refusals and sizes of kda_lin_* and kda_qk_rope* (no GPU: every check runs before any HIP call, the fake pointers
are never dereferenced), and the frequency tables."""
import ctypes
import math

import numpy as np
import pytest
import torch

from gated_delta_rule_86_amd import kda, linattn, qkrope

STEP = 1 << 30
BASE = 1 << 40


def ptr(i):
    return BASE + i * STEP


def lin_args(**ch):
    a = dict(q=ptr(0), k=ptr(1), v=ptr(2), decay=ptr(3), per_token=1, scale=0.1, out=ptr(4), h0=ptr(5), h0_dt=2,
             ht=ptr(6), ht_dt=2, cu=None, cu_host=None, B=2, T=100, Hk=2, H=4, N=0, K=128, V=128, strides=None,
             ws=ptr(7), ws_bytes=1 << 28)
    a.update(ch)
    if a["strides"] is not None:
        a["strides"] = (ctypes.c_int64 * len(a["strides"]))(*a["strides"])
    if a["cu_host"] is not None:
        a["cu_host"] = np.array(a["cu_host"], dtype=np.int64)
    return a


def lin_call(name="kda_lin_fwd", **ch):
    a = lin_args(**ch)
    host = None if a["cu_host"] is None else a["cu_host"].ctypes.data
    return getattr(kda.lib(), name)(a["q"], a["k"], a["v"], a["decay"], a["per_token"], a["scale"], a["out"], a["h0"],
                                    a["h0_dt"], a["ht"], a["ht_dt"], a["cu"], host, a["B"], a["T"], a["Hk"], a["H"],
                                    a["N"], a["K"], a["V"], a["strides"], a["ws"], a["ws_bytes"], None)


LIN_ERRORS = [
    (1, dict(q=None)), (1, dict(k=None)), (1, dict(v=None)), (1, dict(decay=None)), (1, dict(out=None)),
    (1, dict(decay=None, per_token=0, T=0)),
    (2, dict(B=0)), (2, dict(T=-1)), (2, dict(H=0, Hk=1)), (2, dict(N=3)), (2, dict(cu=ptr(8), N=2)),
    (2, dict(B=1, cu=ptr(8), N=0)), (2, dict(T=1 << 36)), (2, dict(B=1 << 29, T=1, H=64)),
    (2, dict(B=1, cu=ptr(8), N=1 << 28, H=4)), (2, dict(T=1 << 34, H=1 << 16, Hk=1)),
    (3, dict(K=64)), (3, dict(V=256)),
    (4, dict(h0_dt=1)), (4, dict(h0_dt=3)), (4, dict(h0=None)), (4, dict(ht_dt=0)),
    (6, dict(scale=float("nan"))), (6, dict(scale=float("inf"))),
    (7, dict(q=ptr(0) + 8)), (7, dict(out=ptr(4) + 2)), (7, dict(decay=ptr(3) + 2)), (7, dict(ws=ptr(7) + 128)),
    (7, dict(h0=ptr(5) + 8)), (7, dict(B=1, cu=ptr(8) + 4, N=2)),
    (11, dict(out=ptr(0))), (11, dict(out=ptr(2))), (11, dict(ht=ptr(1))), (11, dict(ht=ptr(5) + 4096)),
    (11, dict(out=ptr(5))), (11, dict(ws=ptr(2))), (11, dict(out=ptr(3))), (11, dict(ht=ptr(4))),
    (12, dict(per_token=2)),
    (14, dict(H=3)), (14, dict(Hk=0)), (14, dict(Hk=8)),
    (15, dict(strides=[8, 4, 128] * 3)), (15, dict(strides=[0, -8, 128] * 3)), (15, dict(strides=[0, 1 << 25, 128] * 3)),
    (15, dict(strides=[0, 256, 128, 0, 256, 128, 0, 512, 100])), (15, dict(strides=[0, 0, 0] * 3)),
    (15, dict(strides=[0, 120, 128] * 3)),
    (9, dict(B=1, cu=ptr(8), N=2, cu_host=[0, 50, 99])), (9, dict(B=1, cu=ptr(8), N=2, cu_host=[1, 50, 100])),
    (9, dict(B=1, cu=ptr(8), N=2, cu_host=[0, 101, 100])),
]


@pytest.mark.parametrize("code,change", LIN_ERRORS, ids=str)
@pytest.mark.parametrize("name", ["kda_lin_fwd", "kda_lin_fwd_recurrent"])
def test_lin_forward_refusals(name, code, change):
    assert lin_call(name, **change) == code


def test_lin_workspace_refusals():
    for kw in (dict(ws=None), dict(ws_bytes=255)):
        assert lin_call(**kw) == 8
        assert lin_call("kda_lin_fwd_recurrent", B=1, cu=ptr(8), N=2, **kw) == 8
    need = linattn.workspace_size(1, 4096, 2)
    assert lin_call(B=1, T=4096, H=2, ws_bytes=need - 1) == 8


def bwd_call(**ch):
    a = lin_args(dout=ptr(9), dht=ptr(10), dq=ptr(11), dk=ptr(12), dv=ptr(13), dd=ptr(14), dh0=ptr(15))
    a.update(ch)
    if a["strides"] is not None:
        a["strides"] = (ctypes.c_int64 * len(a["strides"]))(*a["strides"])
    return kda.lib().kda_lin_bwd(a["q"], a["k"], a["v"], a["decay"], a["per_token"], a["scale"], a["h0"], a["h0_dt"],
                                 a["dout"], a["dht"], a["dq"], a["dk"], a["dv"], a["dd"], a["dh0"], a["cu"], None,
                                 a["B"], a["T"], a["Hk"], a["H"], a["N"], a["K"], a["V"], a["strides"], a["ws"],
                                 a["ws_bytes"], None)


@pytest.mark.parametrize("code,change", [
    (1, dict(dout=None)), (1, dict(dq=None)), (1, dict(dv=None)), (1, dict(decay=None)), (2, dict(B=0)),
    (3, dict(K=64)), (4, dict(h0_dt=0)), (6, dict(scale=float("nan"))), (7, dict(dout=ptr(9) + 8)),
    (7, dict(dk=ptr(12) + 8)), (7, dict(dd=ptr(14) + 1)), (7, dict(dh0=ptr(15) + 4)), (12, dict(per_token=-1)),
    (11, dict(dq=ptr(0))), (11, dict(dq=ptr(9))), (11, dict(dk=ptr(11))), (11, dict(dh0=ptr(10))), (11, dict(dd=ptr(3))),
    (11, dict(dh0=ptr(5))), (11, dict(ws=ptr(13))), (14, dict(H=5)), (15, dict(strides=[0, 4, 128] * 3)),
    (8, dict(ws=None)), (8, dict(ws_bytes=1024)),
], ids=str)
def test_lin_backward_refusals(code, change):
    assert bwd_call(**change) == code


def test_lin_workspace_sizes():
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    # enough rows x heads, or too short to cut: the status word alone
    for B, T, H in [(64, 4096, 8), (1, 64, 4), (3, 0, 2), (1, 500, 1)]:
        assert linattn.workspace_size(B, T, H) == 256
    # cut rows: a state and a factor for each segment and head
    for B, T, H, N, varlen in [(1, 4096, 4, 0, False), (2, 4096, 16, 0, False), (1, 30000, 8, 9, True)]:
        got = linattn.workspace_size(B, T, H, N, varlen)
        slots = (got - 256) // (65536 + 4) // H * H
        assert slots > 0 and got == 256 + up(slots * 65536) + up(slots * 4), (B, T, H)
    assert linattn.workspace_size(0, 10, 1) == 0 and linattn.workspace_size(2, 10, 1, 3, True) == 0
    assert linattn.bwd_workspace_size(1, 64, 2, 3) == 0  # heads
    shared, alone = linattn.bwd_workspace_size(4, 100, 2, 4, need_ddecay=False), linattn.bwd_workspace_size(
        4, 100, 4, 4, need_ddecay=False)
    assert shared - alone == 2 * 4 * 100 * 4 * 512 and alone == 256
    assert linattn.bwd_workspace_size(4, 100, 4, 4) > alone


def test_launch_limits():
    """Sizes whose launch would hold 2^32 threads or more are refused by the checks, not by the runtime."""
    assert linattn.workspace_size((1 << 21) - 2, 1, 4) == 256 and linattn.workspace_size(1 << 21, 1, 4) == 0
    assert linattn.bwd_workspace_size(1 << 17, 1024, 4, 4) == 0  # the scan over two segments a row
    assert linattn.bwd_workspace_size(1 << 17, 1024, 4, 4, need_ddecay=False) == 256
    alone = dict(B=1, T=100, cu=ptr(8), h0=None, h0_dt=0, ht=None, ht_dt=0)
    assert lin_call("kda_lin_fwd_recurrent", N=1 << 22, **alone) == 2
    assert lin_call("kda_lin_fwd_recurrent", N=1 << 21, ws_bytes=255, **alone) == 8
    rope = kda.lib().kda_qk_rope_bwd_workspace_size
    assert rope(1, 1 << 30, 1, 1, 16) == 0 and rope(1, (1 << 30) - 64, 1, 1, 16) == 1024 * 16 * 4


@pytest.mark.parametrize("B,H,code", [((1 << 21) - 2, 4, 11), (1 << 21, 4, 11), (3 << 20, 4, 11), ((1 << 22) - 2, 4, 11), (1 << 22, 4, 2),
                                      ((1 << 24) - 8, 1, 11), (1 << 24, 1, 2), (1 << 21, 8, 2)])
@pytest.mark.parametrize("T", [1, 9])
def test_token_by_token_limit_without_cu_seqlens(B, H, code, T):
    """The limit is sequences x heads of 2^24, with and without cu_seqlens.  out overlaps q in these calls, so that sizes within
    the limit end in KDA_ERR_ALIAS, before anything could be launched."""
    alone = dict(out=ptr(0), h0=None, h0_dt=0, ht=None, ht_dt=0, ws=None, ws_bytes=0, Hk=1)
    assert lin_call("kda_lin_fwd_recurrent", B=B, T=T, H=H, **alone) == code


def rope_call(back=False, **ch):
    a = dict(q=ptr(0), k=ptr(1), y=[ptr(2), ptr(3)], g=[ptr(4), ptr(5)], wq=ptr(6), wk=ptr(7), f=ptr(8), pos=ptr(9),
             dwq=ptr(10), dwk=ptr(11), B=2, T=10, Hq=4, Hk=2, D=128, R=64, dtype=1, norm=1, eps=1e-6, inter=0, m=1.0,
             strides=None, ws=ptr(12), ws_bytes=1 << 24)
    a.update(ch)
    if back and a["strides"] is not None and len(a["strides"]) == 12:  # gradients of the outputs laid out as q, k
        a["strides"] = a["strides"][:6] * 2 + a["strides"][6:]
    st = None if a["strides"] is None else (ctypes.c_int64 * len(a["strides"]))(*a["strides"])
    sizes = (a["B"], a["T"], a["Hq"], a["Hk"], a["D"], a["R"], a["dtype"], a["norm"], a["eps"], a["inter"], a["m"], st)
    if back:
        return kda.lib().kda_qk_rope_bwd(a["q"], a["k"], *a["g"], *a["y"], a["wq"], a["wk"], a["dwq"], a["dwk"], a["f"],
                                         a["pos"], *sizes, a["ws"], a["ws_bytes"], None)
    return kda.lib().kda_qk_rope(a["q"], a["k"], *a["y"], a["wq"], a["wk"], a["f"], a["pos"], *sizes, None)


# q and k as views of one buffer, row by row: heads of q, then of k
FUSED = [10 * 768, 768, 128]


@pytest.mark.parametrize("code,change", [
    (1, dict(q=None)), (1, dict(k=None)), (1, dict(y=[None, ptr(3)])), (1, dict(f=None)),
    (2, dict(B=0)), (2, dict(T=-1)), (2, dict(Hq=0)), (2, dict(Hk=0)), (2, dict(T=1 << 31)), (2, dict(Hq=5000)),
    (16, dict(D=120)), (16, dict(D=1024)), (16, dict(D=0, R=0)), (16, dict(R=24)), (16, dict(R=256)), (16, dict(R=-16)),
    (4, dict(dtype=0)), (4, dict(dtype=4)), (12, dict(norm=3)), (12, dict(norm=-1)), (12, dict(inter=2)),
    (6, dict(eps=-1.0)), (6, dict(eps=float("nan"))), (6, dict(m=float("inf"))),
    (7, dict(q=ptr(0) + 8)), (7, dict(y=[ptr(2), ptr(3) + 2])), (7, dict(wq=ptr(6) + 2)), (7, dict(pos=ptr(9) + 4)),
    (11, dict(y=[ptr(1), ptr(3)])), (11, dict(y=[ptr(2), ptr(2)])), (11, dict(y=[ptr(0) + 16, ptr(3)])),
    (11, dict(y=[ptr(6), ptr(3)])), (11, dict(y=[ptr(9), ptr(3)])),
    (15, dict(strides=[4, 512, 128] * 4)), (15, dict(strides=[-8, 512, 128] * 4)),
    # outputs whose heads or rows overlap themselves
    (11, dict(strides=[5120, 512, 128, 2560, 256, 128, 5120, 512, 64, 2560, 256, 128])),
    (11, dict(strides=[5120, 512, 128, 2560, 256, 128, 5120, 256, 128, 2560, 256, 128])),
    # in place on one buffer, but k's heads lie where q's are
    (11, dict(q=ptr(0), k=ptr(0) + 256, y=[ptr(0), ptr(0) + 256], strides=FUSED * 4)),
], ids=str)
@pytest.mark.parametrize("back", [False, True])
def test_rope_refusals(back, code, change):
    assert rope_call(back, **change) == code


@pytest.mark.parametrize("code,change", [
    (1, dict(g=[None, ptr(5)])), (1, dict(wq=None)), (7, dict(dwq=ptr(10) + 1)), (7, dict(ws=ptr(12) + 16)),
    (11, dict(dwq=ptr(0))), (11, dict(dwq=ptr(11))), (11, dict(ws=ptr(2))), (11, dict(dwk=ptr(7))),
    (8, dict(ws=None)), (8, dict(ws_bytes=100)),
], ids=str)
def test_rope_backward_refusals(code, change):
    assert rope_call(True, **change) == code


def test_rope_allows_views_of_one_buffer():
    """q and k interleaved in one buffer, replaced in place: passes every check up to a later refusal (the
    workspace's in the backward pass, which is looked at last)."""
    ok = dict(q=ptr(0), k=ptr(0) + 1024, y=[ptr(0), ptr(0) + 1024], strides=FUSED * 4, ws=None)
    assert rope_call(True, **ok) == 8
    one = dict(ok, T=1, B=5, strides=[768, 0, 128] * 4)  # one token per row: rows follow the batch
    assert rope_call(True, **one) == 8
    assert rope_call(True, **dict(one, k=ptr(0) + 512, y=[ptr(0), ptr(0) + 512])) == 11


@pytest.mark.parametrize("B,T", [(1, 10), (2, 10), (3, 1), (1, 1)])
@pytest.mark.parametrize("Hq,Hk", [(4, 2), (1, 1), (3, 1)])
def test_rope_allows_any_order_of_dimensions(B, T, Hq, Hk):
    """Outputs laid out [B, heads, T, D], [T, B, heads, D] or [heads, B, T, D] share no byte with themselves; q and k side by side in one
    buffer of any of these may be replaced in place, and k's place must still be clear of q's."""
    D, H = 128, Hq + Hk
    for q_st, k_st in (([Hq * T * D, D, T * D], [Hk * T * D, D, T * D]), ([Hq * D, B * Hq * D, D], [Hk * D, B * Hk * D, D]),
                       ([T * D, D, B * T * D], [T * D, D, B * T * D])):
        st = [T * Hq * D, Hq * D, D, T * Hk * D, Hk * D, D] + q_st + k_st
        assert rope_call(True, B=B, T=T, Hq=Hq, Hk=Hk, strides=st, ws=None) == 8
    for one, at in (([H * T * D, D, T * D], Hq * T * D), ([H * D, B * H * D, D], Hq * D), ([T * D, D, B * T * D], Hq * B * T * D)):
        ok = dict(B=B, T=T, Hq=Hq, Hk=Hk, strides=one * 4, ws=None)
        for off, code in ((2 * at, 8), (2 * at - 2 * D, 11)):
            p = [ptr(0), ptr(0) + off]
            assert rope_call(True, **ok, q=p[0], k=p[1], y=p) == code
        # the other way round: k's heads first
        p = [ptr(0) + 2 * (at // Hq * Hk), ptr(0)]
        assert rope_call(True, **ok, q=p[0], k=p[1], y=p) == 8


def test_rope_views_against_brute_force():
    """Random small layouts of two outputs: never accepted when they share a byte, with each other or with themselves."""
    rng = np.random.default_rng(0)
    D, accepted, clear = 16, 0, 0
    for _ in range(3000):
        B, T, Hq, Hk = (int(x) for x in rng.integers(1, 4, 4))
        st = [int(x) * 8 for x in rng.integers(0, 13, 6)]
        base = int(rng.integers(0, 24)) * 8
        place = lambda o, s, H: [o + b * s[0] + t * s[1] + h * s[2] + c for b in range(B) for t in range(T)  # noqa: E731
                                 for h in range(H) for c in range(D)]
        both = place(0, st[:3], Hq) + place(base, st[3:], Hk)
        free = len(set(both)) == len(both)
        y = [ptr(4), ptr(4) + 2 * base]
        full = [T * Hq * D, Hq * D, D, T * Hk * D, Hk * D, D]
        code = rope_call(True, B=B, T=T, Hq=Hq, Hk=Hk, D=D, R=16, strides=full * 2 + st, y=y, g=[ptr(2), ptr(3)], ws=None)
        assert code in (8, 11) and (free or code == 11)
        accepted, clear = accepted + (code == 8), clear + free
    assert accepted > 0.5 * clear > 20


def test_python_refusals():
    """What the bindings refuse before the library is called."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    q, k, v, d, out = z(1, 4, 2, 128), z(1, 4, 2, 128), z(1, 4, 4, 128), z(4, dt=torch.float32), z(1, 4, 4, 128)
    for bad in (dict(q=z(1, 4, 256)), dict(q=q.float()), dict(k=z(1, 5, 2, 128)), dict(v=z(1, 5, 4, 128)),
                dict(d=z(3, dt=torch.float32)), dict(d=z(4)), dict(d=z(1, 4, 4, dt=torch.float32).mT), dict(out=z(1, 4, 4, 64)),
                dict(out=out.float()), dict(q=z(1, 4, 2, 256)[..., ::2])):
        a = dict(q=q, k=k, v=v, d=d, out=out) | bad
        with pytest.raises(ValueError):
            linattn.fwd(a["q"], a["k"], a["v"], a["d"], 1.0, a["out"])
    s = z(1, 4, 128, 128, dt=torch.float32)
    for kw in (dict(initial_state=s[:, :2]), dict(initial_state=s.half()), dict(initial_state=s, final_state=s.bfloat16()),
               dict(final_state=s.mT), dict(cu_seqlens=torch.zeros(2, dtype=torch.int32)),
               dict(cu_seqlens_host=[0, 4])):
        with pytest.raises(ValueError):
            linattn.fwd(q, k, v, d, 1.0, out, **kw)
    with pytest.raises(ValueError):
        linattn.bwd(q, k, v, d, 1.0, out.float())
    with pytest.raises(ValueError):
        linattn.bwd(q, k, v, d, 1.0, out, dfinal_state=s.bfloat16())
    x, y, f = z(1, 4, 2, 64), z(1, 4, 1, 64), z(32, dt=torch.float32)
    p = torch.zeros(1, 4, dtype=torch.int64)
    for a in ((x, y, p.int(), f, x, y), (x, y, p[:, :2], f, x, y), (x, y, p, f.double(), x, y), (x, y.float(), p, f, x, y),
              (x, y, p, f, y, y), (x[0], y, p, f, x, y), (x.double(), y.double(), p, f, x.double(), y.double())):
        with pytest.raises(ValueError):
            qkrope.fwd(*a)
    for kw in (dict(norm="layer"), dict(q_weight=z(64)), dict(k_weight=z(32, dt=torch.float32))):
        with pytest.raises(ValueError):
            qkrope.fwd(x, y, p, f, x, y, **kw)


def test_stream_of_another_device_is_refused():
    import types
    there = types.SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=7)
    assert linattn._raw_stream(there, 1) == qkrope._raw_stream(there, 1) == 7
    with pytest.raises(ValueError, match="cuda:0"):
        linattn._raw_stream(there, 0)


def test_frequencies():
    f, m = qkrope.inv_freq(64, 10000.0)
    want = [10000.0 ** (-2 * i / 64) for i in range(32)]
    assert m == 1.0 and torch.equal(f, torch.tensor(want, dtype=torch.float64).float())
    g, _ = qkrope.inv_freq(64, scaling="linear", factor=4.0)
    assert torch.allclose(g, f / 4, rtol=2.0 ** -23)
    g, _ = qkrope.inv_freq(64, scaling="ntk", factor=8.0)
    assert g[0] == f[0] and math.isclose(float(g[-1]), float(f[-1]) / 8, rel_tol=1e-6) and (g <= f).all()
    g, m = qkrope.inv_freq(128, scaling="yarn", factor=16.0, original_context=4096)
    f, _ = qkrope.inv_freq(128)
    turns = f.double() * 4096 / (2 * math.pi)
    assert math.isclose(m, 0.1 * math.log(16) + 1)
    assert torch.equal(g[turns > 40], f[turns > 40])                       # quick pairs stay
    assert torch.allclose(g[turns < 0.8], f[turns < 0.8] / 16, rtol=1e-6)  # slow ones are stretched whole
    assert (g <= f).all() and (g >= f / 16 * (1 - 1e-6)).all() and (g[1:] <= g[:-1]).all()
    for bad in (dict(scaling="other"), dict(scaling="yarn"), dict(factor=0.5), dict(base=1.0)):
        with pytest.raises(ValueError):
            qkrope.inv_freq(64, **bad)
    with pytest.raises(ValueError):
        qkrope.inv_freq(7)
    assert qkrope.inv_freq(0)[0].numel() == 0


@pytest.mark.parametrize("R,base", [(32, 1e4), (64, 1e4), (128, 1e4), (128, 5e5)])
@pytest.mark.parametrize("context", [256, 4096, 32768, 65536, 131072, 1 << 20])
def test_yarn_ramp_ends_where_its_pairs_do(R, base, context):
    """The ramp runs between the (real) indices of the pairs that turn 32 times and once over the original context, and may end
    behind the last pair: a pair that still turns more than once is not divided by the whole factor."""
    factor = 4.0
    f, _ = qkrope.inv_freq(R, base, scaling="yarn", factor=factor, original_context=context)
    i = np.arange(R // 2, dtype=np.float64)
    plain = base ** (-2 * i / R)
    index = lambda turns: R * math.log(context / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(index(32.0)), 0), min(math.ceil(index(1.0)), R - 1)
    keep = 1.0 - np.clip((i - lo) / (hi - lo), 0.0, 1.0)
    want = plain * keep + plain / factor * (1.0 - keep)
    got = f.double().numpy()
    np.testing.assert_allclose(got, want, rtol=2.0 ** -23)
    turns = context * plain / (2 * math.pi)
    assert (np.abs(got / plain - 1.0)[turns >= 32.0] < 2.0 ** -22).all()
    assert (np.abs(got / plain * factor - 1.0)[turns <= 1.0] < 2.0 ** -22).all()
    between = (turns > 1.0) & (i > lo) & (i < hi)
    assert (got[between] > plain[between] / factor * 1.001).all() and (got[between] < plain[between]).all()
