"""The int32 and fp32 tables of the token calls are aligned to their elements, or refused, and so are
sizes past 32 bits (on the CPU; pointers here are never followed)."""
import pytest

import routed_expert_ffn_02_amd as R
from test_frame_refusals import A, LONG, combine_backward, dispatch, move, topk


@pytest.mark.parametrize("shape", [{}, dict(T=2000, k=4), LONG])
@pytest.mark.parametrize("table", [dict(idx=A[0] + 2), dict(perm=A[3] + 1), dict(inv=A[4] + 2), dict(off=A[5] + 3)])
def test_dispatch(table, shape):
    assert dispatch(**shape, **table) == R.MOE_EINVAL
    assert dispatch(**shape, **table, x=None, xs=None) == R.MOE_EINVAL     # the sort alone


@pytest.mark.parametrize("off", [1, 2, 3])
def test_moves(off):
    assert move("back", inv=A[1] + off) == R.MOE_EINVAL
    assert move("combine", inv=A[1] + off) == R.MOE_EINVAL
    assert move("combine", w=A[3] + off) == R.MOE_EINVAL
    for table in (dict(inv=A[2] + off), dict(w=A[3] + off), dict(dw=A[5] + off), dict(w=A[3] + off, dw=None),
                  dict(dw=A[5] + off, dys=None)):
        assert combine_backward(**table) == R.MOE_EINVAL


@pytest.mark.parametrize("off", [1, 2, 3])
def test_topk_backward(off):
    for table in (dict(z=A[0] + off), dict(idx=A[1] + off), dict(dw=A[2] + off), dict(dz=A[3] + off),
                  dict(z=A[0] + off, dz=A[0] + off)):
        assert topk(**table) == R.MOE_EINVAL


@pytest.mark.parametrize("past", [1 << 31, 1 << 32, -(1 << 32), 1 << 63])
def test_workspace_sizes_past_32_bits(past):
    for f, sizes in ((R.moe_dispatch_workspace, (5000, 8, 16)), (R.moe_block_norm_workspace, (64, 128))):
        assert f(*sizes) > 0
        for i in range(len(sizes)):
            with pytest.raises(R.MoeError) as e:
                f(*[v + past * (i == j) for j, v in enumerate(sizes)])
            assert e.value.status == R.MOE_EINVAL and f.__name__ in str(e.value)
    with pytest.raises(R.MoeError):
        R.moe_block_norm_workspace(4, 8193)
