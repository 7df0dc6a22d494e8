"""Outputs of kda_gated_norm and kda_residual_norm in the place of a broadcast input (no GPU: the calls are refused before any HIP
call, the fake pointers are never dereferenced)."""
import pytest

from test_gdn_norm_host import gated_call, ptr, residual_call

ALIAS = 11


@pytest.mark.parametrize("sizes", [dict(), dict(B=1), dict(T=1), dict(H=1), dict(B=1, T=1), dict(T=1, H=1), dict(B=1, H=1)], ids=str)
@pytest.mark.parametrize("dtype", [1, 2, 3])
@pytest.mark.parametrize("which", ["x", "gate"])
def test_gated_norm_in_the_place_of_one_row(sizes, dtype, which):
    """One row broadcast over all others is not contiguous: they read it while the first row of out is written over it."""
    one, all_rows = [0, 0, 0], [5120, 512, 128]
    if sizes.get("H") == 1:
        all_rows = [1280, 128, 128]
    strides = one + all_rows if which == "x" else all_rows + one
    assert gated_call(y=ptr(0 if which == "x" else 1), strides=strides, dtype=dtype, **sizes) == ALIAS


@pytest.mark.parametrize("sizes", [dict(), dict(B=1), dict(T=1)], ids=str)
@pytest.mark.parametrize("dtype,rdtype", [(1, 1), (1, 2), (2, 2), (3, 2)])
def test_residual_norm_in_the_place_of_one_row(sizes, dtype, rdtype):
    kw = dict(dtype=dtype, rdtype=rdtype, **sizes)
    assert residual_call(y=ptr(0), strides=[0, 0, 1280, 128], **kw) == ALIAS
    assert residual_call(zo=ptr(1), strides=[1280, 128, 0, 0], **kw) == ALIAS


def test_rows_broadcast_over_one_dimension():
    assert gated_call(y=ptr(0), strides=[5120, 512, 0, 5120, 512, 128]) == ALIAS
    assert gated_call(y=ptr(1), strides=[5120, 512, 128, 5120, 0, 128]) == ALIAS
    assert gated_call(y=ptr(0), strides=[0, 512, 128, 5120, 512, 128]) == ALIAS
    assert residual_call(y=ptr(0), strides=[1280, 0, 1280, 128]) == ALIAS
    assert residual_call(zo=ptr(1), strides=[1280, 128, 0, 128]) == ALIAS
