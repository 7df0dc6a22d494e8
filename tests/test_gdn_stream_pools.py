"""stream= of the gated delta rule and the norms: what a call allocates comes from the pool of the stream that its kernels run on, on the
stand-ins of test_stream_pools."""
import contextlib

import pytest
import torch

from gated_delta_rule_86_amd import blocknorm, gdn

from test_stream_pools import D, stands  # noqa: F401


@pytest.fixture
def here(stands, monkeypatch):  # noqa: F811
    from gated_delta_rule_86_amd import kda
    for m in (gdn, blocknorm):
        monkeypatch.setattr(m, "lib", kda.lib)
        monkeypatch.setattr(m, "_gpu_index", lambda x: 0)
        monkeypatch.setattr(m, "_On", lambda i: contextlib.nullcontext())
        monkeypatch.setattr(m, "_raw_stream", lambda s, i: 0)
    return stands


def calls():
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    x, g, h = z(1, 3, 2, D), z(1, 3, 2, dtype=torch.float32), z(1, 2, D, D, dtype=torch.float32)
    y, w = z(1, 3, D), z(D, dtype=torch.float32)
    cu = torch.tensor([0, 3])
    return {
        "gdn.fwd": lambda **k: gdn.fwd(x, x, x, g, g, 1.0, x, None, h, **k),
        "gdn.fwd_recurrent": lambda **k: gdn.fwd_recurrent(x, x, x, g, g, 1.0, x, None, h, cu, **k),
        "gdn.bwd": lambda **k: gdn.bwd(x, x, x, g, g, 1.0, x, **k),
        "blocknorm.gated_bwd": lambda **k: blocknorm.gated_bwd(x, x, x, weight=w, **k),
        "blocknorm.residual_bwd": lambda **k: blocknorm.residual_bwd(y, y, y, weight=w, scale=w, **k),
    }


ALLOCATING = sorted(calls())


@pytest.mark.parametrize("name", ALLOCATING)
def test_blocks_come_from_the_streams_own_pool(here, name):
    calls()[name](stream=here.side)
    assert here.blocks and here.current is here.home
    for b in here.blocks:
        assert b.pool is here.side
        assert any(s is here.home for s in b.users)


@pytest.mark.parametrize("name", ALLOCATING)
def test_current_stream(here, name):
    for stream in (None, here.home):
        calls()[name](stream=stream)
    assert here.blocks and all(b.pool is here.home and not b.users for b in here.blocks)
