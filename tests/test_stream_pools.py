"""stream=: what a call allocates must come from the pool of the stream that its kernels run on.  A block of the current stream's pool may
have been freed while that stream's work on it is still pending, and nothing orders `stream` behind that work.

The CPU tests run the bindings on stand-ins for the library, the streams and torch.empty, and note in whose pool each block was
allocated; the GPU tests look at the addresses."""
import contextlib
import types

import pytest
import torch

from gated_delta_rule_86_amd import kda, linattn, qkrope

D = 128


class Block:
    def __init__(self, pool, shape):
        self.pool, self.shape, self.users = pool, shape, []

    def data_ptr(self):
        return 1 << 30

    device = torch.device("cuda:0")

    def numel(self):
        return torch.Size(self.shape).numel()

    def element_size(self):
        return 1

    def is_contiguous(self):
        return True

    def record_stream(self, s):
        self.users.append(s)


@pytest.fixture
def stands(monkeypatch):
    """current: the current stream; blocks: everything allocated, with the stream current at that time."""
    t = types.SimpleNamespace(current=types.SimpleNamespace(cuda_stream=1, device=torch.device("cuda:0")), blocks=[])
    t.home = t.current
    t.side = types.SimpleNamespace(cuda_stream=2, device=torch.device("cuda:0"))

    @contextlib.contextmanager
    def stream(s):
        old, t.current = t.current, s
        yield
        t.current = old

    def empty(*shape, **kw):
        shape = shape[0] if isinstance(shape[0], (tuple, list, torch.Size)) else shape
        t.blocks.append(Block(t.current, shape))
        return t.blocks[-1]

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 4096 if name.endswith("workspace_size") else 0

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: t.current)
    monkeypatch.setattr(torch, "empty", empty)
    for m in (kda, linattn, qkrope):
        monkeypatch.setattr(m, "lib", Lib)
    for m in (linattn, qkrope):
        monkeypatch.setattr(m, "_gpu_index", lambda x: 0)
        monkeypatch.setattr(m, "_On", lambda i: contextlib.nullcontext())
        monkeypatch.setattr(m, "_raw_stream", lambda s, i: 0)
    return t


def calls():
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    x, beta, h = z(1, 3, 2, D), z(1, 3, 2), z(1, 2, D, D, dtype=torch.float32)
    d, a, bias = z(2, dtype=torch.float32), z(2, dtype=torch.float32), z(2, D, dtype=torch.float32)
    cu = torch.tensor([0, 3])
    f, w = z(D // 2, dtype=torch.float32), z(D, dtype=torch.float32)
    return {
        "kda.fwd": lambda **k: kda.fwd(x, x, x, x, beta, 1.0, x, a, bias, -5.0, **k),
        "kda.fwd_recurrent": lambda **k: kda.fwd_recurrent(x, x, x, x, beta, 1.0, x, a, bias, -5.0, **k),
        "kda.bwd": lambda **k: kda.bwd(x, x, x, x, beta, 1.0, a, bias, -5.0, x, **k),
        "kda.chunk_table": lambda **k: kda.chunk_table(cu, 1, 3, 2, **k),
        "linattn.fwd": lambda **k: linattn.fwd(x, x, x, d, 1.0, x, None, h, **k),
        "linattn.fwd_recurrent": lambda **k: linattn.fwd_recurrent(x, x, x, d, 1.0, x, None, h, cu, **k),
        "linattn.bwd": lambda **k: linattn.bwd(x, x, x, d, 1.0, x, **k),
        "qkrope.bwd": lambda **k: qkrope.bwd(x, x, None, f, x, x, q_weight=w, k_weight=w, **k),
    }


ALLOCATING = sorted(calls())


@pytest.mark.parametrize("name", ALLOCATING)
def test_blocks_come_from_the_streams_own_pool(stands, name):
    calls()[name](stream=stands.side)
    assert stands.blocks and stands.current is stands.home
    for b in stands.blocks:
        assert b.pool is stands.side                # what was freed there is ordered before the kernels
        assert any(s is stands.home for s in b.users)  # and the caller's own use of results before their next life


@pytest.mark.parametrize("name", ALLOCATING)
def test_current_stream(stands, name):
    for stream in (None, stands.home):
        calls()[name](stream=stream)
    assert stands.blocks and all(b.pool is stands.home and not b.users for b in stands.blocks)


@pytest.mark.gpu
def test_a_block_freed_on_the_current_stream_is_not_taken():
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(0)
    n = lambda *s: torch.randn(s, generator=g, device=dev).bfloat16()  # noqa: E731
    T = 3000
    q, k, v, do = (n(1, T, 1, D) for _ in range(4))
    d, f = torch.full((1,), -0.01, device=dev), torch.ones(D // 2, device=dev)
    out, w = torch.empty_like(v), torch.ones(D, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = linattn.bwd(q, k, v, d, D ** -0.5, do)
    for call in (lambda: {"workspace": linattn.fwd(q, k, v, d, D ** -0.5, out, stream=side)},
                 lambda: linattn.bwd(q, k, v, d, D ** -0.5, do, stream=side),
                 lambda: qkrope.bwd(q, k, None, f, q, k, q_weight=w, k_weight=w, stream=side)):
        r = call()  # its sizes
        torch.cuda.synchronize()
        freed = [torch.empty(x.shape, dtype=x.dtype, device=dev) for x in r.values() for _ in range(3)]
        spans = [(x.data_ptr(), x.data_ptr() + x.numel() * x.element_size()) for x in freed]
        del freed
        r = call()
        torch.cuda.synchronize()
        for x in r.values():
            lo, hi = x.data_ptr(), x.data_ptr() + x.numel() * x.element_size()
            assert not any(lo < b and a < hi for a, b in spans)
        if "dv" in r:
            assert all(torch.equal(r[m], want[m]) for m in ("dq", "dk", "dv", "ddecay"))
