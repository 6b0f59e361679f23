"""The experts' products with the most rows at the largest strides, on the CPU: 2^26 rows 2^36 elements apart reach past
64 bits of bytes, where blocks that lie in each other would seem apart."""
import ctypes

import pytest

import routed_expert_ffn_02_amd as R

L = R.lib
F32, BF16 = R.MOE_AFMT_F32, R.MOE_AFMT_BF16
A = [0x100_0000_0000 * (i + 1) for i in range(16)]
FAR, ROWS = 1 << 36, 1 << 26


def config(fmt, **kw):
    a = dict(rows=ROWS, n_experts=1, K=32, N=32, fmt=fmt, y_fmt=fmt, dw_fmt=fmt, act=R.MOE_ACT_SILU, ld_x=0, ld_dx=0, ld_w=0, gs_w=0,
             ld_y=0, ld_residual=0, ld_z=0)
    a.update(kw)
    return ctypes.byref(R.moe_product_config(*a.values()))


@pytest.mark.parametrize("fmt", [F32, BF16])
@pytest.mark.parametrize("ld", [FAR, FAR - 64, FAR // 2, FAR // 2 + 1, FAR // 4 + 32])
def test_blocks_in_each_other_are_refused(fmt, ld):
    n = 1 << 62
    both = config(fmt, ld_x=ld, ld_y=ld)
    assert L.moe_glu(both, A[0], A[1], None, A[0], None, None) == R.MOE_EINVAL
    assert L.moe_linear(both, A[0], A[1], None, None, None, A[0], None, None) == R.MOE_EINVAL
    assert L.moe_linear(config(fmt, ld_y=ld, ld_residual=ld), A[0], A[1], None, A[2], None, A[2] + 64, None, None) == R.MOE_EINVAL
    assert L.moe_linear(config(fmt, ld_y=ld, ld_z=ld), A[0], A[1], None, None, None, A[2], A[2], None) == R.MOE_EINVAL
    grads = config(fmt, ld_x=ld, ld_dx=ld, ld_y=ld, ld_z=ld)
    assert L.moe_glu_backward(grads, A[0], A[1], A[2], A[3], None, A[0], A[4], 1 << 63, n, None) == R.MOE_EINVAL
    assert L.moe_linear_backward(grads, A[0], A[1], A[2], A[3], None, A[1], A[4], A[5], 1 << 63, n, None) == R.MOE_EINVAL


@pytest.mark.parametrize("fmt", [F32, BF16])
def test_rows_past_any_memory_are_refused(fmt):
    """Rows whose last one starts 2^58 elements and more behind the first, in every operand."""
    for name in ("ld_x", "ld_y", "ld_z", "ld_residual"):
        assert L.moe_linear(config(fmt, **{name: FAR}), A[0], A[1], None, A[2], None, A[3], A[4], None) == R.MOE_EINVAL, name
    for name in ("ld_x", "ld_dx", "ld_y", "ld_z"):
        assert L.moe_linear_backward(config(fmt, **{name: FAR}), A[0], A[1], A[2], A[3], None, A[4], A[5], None, 1 << 63, 1 << 62,
                                     None) == R.MOE_EINVAL, name
