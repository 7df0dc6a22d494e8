"""q/k norm and rotation through views in any order of dimensions: the same bits as contiguous tensors, nothing else written."""
import pytest
import torch

from gated_delta_rule_86_amd import qkrope

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
ORDERS = {"heads first": (0, 2, 1, 3), "tokens first": (1, 0, 2, 3), "heads outermost": (2, 0, 1, 3)}  # of [B, T, H, D]


def view(buf, order):
    back = [order.index(i) for i in range(4)]
    return buf.permute(back)


@pytest.mark.parametrize("order", ORDERS, ids=str)
@pytest.mark.parametrize("B,T,Hq,Hk", [(2, 37, 4, 2), (1, 1, 3, 1), (5, 1, 2, 2), (1, 300, 1, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_any_order(order, B, T, Hq, Hk, dtype):
    D, order = 64, ORDERS[order]
    g = torch.Generator(device=DEV).manual_seed(T)
    n = lambda *s: torch.randn(s, generator=g, device=DEV).to(dtype)  # noqa: E731
    q, k = n(B, T, Hq, D), n(B, T, Hk, D)
    f, _ = qkrope.inv_freq(D, device=DEV)
    w = n(D).float()
    kw = dict(q_weight=w, k_weight=w)
    want = [torch.empty_like(q), torch.empty_like(k)]
    qkrope.fwd(q, k, None, f, *want, **kw)
    shape = lambda H: [(B, T, H, D)[i] for i in order]  # noqa: E731
    out = [view(torch.full(shape(H), 7.0, dtype=dtype, device=DEV), order) for H in (Hq, Hk)]
    qkrope.fwd(q, k, None, f, *out, **kw)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    # in place, side by side in one buffer with two heads more than are used
    buf = n(*shape(Hq + Hk + 2))
    both = view(buf, order)
    both[:, :, 1:1 + Hq], both[:, :, 1 + Hq:1 + Hq + Hk] = q, k
    before = both.clone()
    x, y = both[:, :, 1:1 + Hq], both[:, :, 1 + Hq:1 + Hq + Hk]
    qkrope.fwd(x, y, None, f, x, y, **kw)
    assert torch.equal(x, want[0]) and torch.equal(y, want[1])
    assert torch.equal(both[:, :, 0], before[:, :, 0]) and torch.equal(both[:, :, -1], before[:, :, -1])
    # gradients read through the same views
    dy = view(n(*shape(Hq + Hk)), order)
    a = qkrope.bwd(view(before.permute(order).contiguous(), order)[:, :, 1:1 + Hq], k, None, f, dy[:, :, :Hq], dy[:, :, Hq:], **kw)
    b = qkrope.bwd(q, k, None, f, dy[:, :, :Hq].contiguous(), dy[:, :, Hq:].contiguous(), **kw)
    assert all(torch.equal(a[m], b[m]) for m in b)
