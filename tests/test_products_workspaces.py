"""Workspaces of the experts' products, on the CPU: what moe_*_workspace gives for a call's sizes is enough for it,
whichever of its outputs it leaves out, and for fewer rows.  (Pointers here are never followed: where nothing is
refused, a call ends at its launch, which fails without a device.)"""
import ctypes
import random

import pytest
import torch

import routed_expert_ffn_02_amd as R

L = R.lib
F32, BF16 = R.MOE_AFMT_F32, R.MOE_AFMT_BF16
A = [0x100_0000_0000 * (i + 1) for i in range(16)]
no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not memory: this runs where nothing can be launched")

# rows, experts, K, N: of projections whose products are too wide to be split along the k, and of narrow ones
SIZES = [(777, 1, 1000, 1001), (5000, 1, 4096, 1024), (4096, 1, 2048, 512), (2048, 1, 2048, 4096), (6144, 32, 2048, 4096), (1, 1, 8, 8),
         (130, 3, 72, 56), (3000, 1, 8, 70)]


def bias_alone(rows, E, K, N, fmt, y_fmt, n, act):
    cfg = R.moe_product_config(rows, E, K, N, fmt, y_fmt, fmt, act, 0, 0, 0, 0, 0, 0, 0)
    return L.moe_linear_backward(ctypes.byref(cfg), A[0], A[1] if act else None, None, None, A[2], None, None, A[3], A[4], n, None)


@no_device
@pytest.mark.parametrize("rows,E,K,N", SIZES)
@pytest.mark.parametrize("fmt", [BF16, F32])
@pytest.mark.parametrize("y_fmt", [BF16, F32])
def test_a_bias_alone_takes_its_sizes_workspace(rows, E, K, N, fmt, y_fmt):
    """As the binding calls it too: without dx and x it knows no K, without an activation only dy's type."""
    n = R.moe_linear_workspace(rows, E, K, N, fmt)
    for act in (R.MOE_ACT_NONE, R.MOE_ACT_GELU):
        assert bias_alone(rows, E, K, N, fmt, y_fmt, n, act) == R.MOE_EHIP
        assert bias_alone(rows, E, 1, N, fmt, y_fmt, n, act) == R.MOE_EHIP
    assert bias_alone(rows, E, 1, N, y_fmt, y_fmt, n, R.MOE_ACT_NONE) == R.MOE_EHIP


@pytest.mark.parametrize("fmt", [BF16, F32])
def test_a_bias_alone_still_needs_its_sums(fmt):
    """3000 rows are summed in 64 parts of 70 columns, 4 bytes each, and 15 bytes reach an alignment."""
    for act in (R.MOE_ACT_NONE, R.MOE_ACT_SILU):
        assert bias_alone(3000, 1, 8, 70, fmt, fmt, 64 * 70 * 4 + 14, act) == R.MOE_EINVAL


@pytest.mark.parametrize("f", [R.moe_glu_workspace, R.moe_linear_workspace])
def test_a_workspace_does_for_fewer_rows(f):
    """A program keeps the workspace of its largest batch: the sums of products split along the k, which the largest one
    may not have, find place in it (140 rows of 3995 and 3819 are not split, 120 are)."""
    rng = random.Random(5)
    for i in range(4000):
        K, N, fmt = rng.randint(1, 4096), rng.randint(1, 4096), rng.choice([F32, BF16])
        E, rows = rng.choice([1, rng.randint(2, 256)]), int(2 ** rng.uniform(0, 14))
        if i == 0:
            E, K, N, fmt, rows = 1, 3995, 3819, BF16, 140
        most = f(rows, E, K, N, fmt)
        for fewer in {120 if i == 0 else rng.randint(1, rows), rng.randint(1, rows), max(rows - 1, 1)}:
            if fewer <= rows:
                assert f(fewer, E, K, N, fmt) <= most, (fewer, rows, E, K, N, fmt)


@no_device
def test_the_calls_take_it():
    n = R.moe_glu_workspace(140, 1, 3995, 3819, BF16)
    cfg = R.moe_product_config(120, 1, 3995, 3819, BF16, BF16, BF16, R.MOE_ACT_SILU, 0, 0, 0, 0, 0, 0, 0)
    assert L.moe_glu_backward(ctypes.byref(cfg), *A[:4], None, A[4], A[5], A[6], n, None) == R.MOE_EHIP
    n = R.moe_linear_workspace(140, 1, 3995, 3819, BF16)
    assert L.moe_linear_backward(ctypes.byref(cfg), *A[:4], None, A[4], A[5], A[6], A[7], n, None) == R.MOE_EHIP
