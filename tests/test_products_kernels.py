"""Which kernels the experts' products take, on the CPU: every one that the library has is reached by a size that the GPU
tests run, so that a change of the rule that chooses them shows here if it leaves one without a test."""
import pytest

import product_launches
from product_sizes import SIZES, case

OURS = {"product_direct", "product", "few_rows", "gradients"}


@pytest.fixture(scope="module")
def stand_in(tmp_path_factory):
    return product_launches.stand_in(tmp_path_factory.mktemp("launch"))


def named(kernel, grid):
    """The kernel, with "cut" behind it where its k is in parts across workgroups."""
    return kernel + (("cut",) if kernel[0] in ("product_direct", "product") and grid[1] > 1 else ())


def test_sizes_take_the_kernels_they_are_for(stand_in):
    cases = [case(row) for row in SIZES]
    _, calls = product_launches.launches(stand_in, [c for c, _ in cases])
    for (c, kernel), (status, ls) in zip(cases, calls):
        assert status == 0, c
        assert kernel in [named(k, grid) for k, grid, _ in ls], (c, kernel, ls)


def test_every_kernel_has_a_size(stand_in):
    """With one weight and over experts."""
    kernels, _ = product_launches.launches(stand_in, [])
    for experts in (False, True):
        reached = {kernel for c, kernel in map(case, SIZES) if (c["E"] > 0) == experts}
        assert {k for k in kernels if k[0] in OURS} == {tuple(v for v in k if v != "cut") for k in reached}
        # gradients of one output are cut along the k by both kinds of kernel, in both types
        assert {(k[0], k[1], k[2]) for k in reached if "cut" in k} == {
            (n, t, op) for n in ("product_direct", "product") for t in ("f32", "bf16") for op in (2, 3)}


def test_launches_are_no_larger_than_counted(stand_in):
    """A launch's threads are counted in 32 bits."""
    _, calls = product_launches.launches(stand_in, [
        dict(call="glu", rows=1 << 23, K=64, N=16384, fmt="bf16"), dict(call="linear_backward", rows=1 << 21, K=65536, N=64, fmt="f32"),
        dict(call="glu_backward", rows=1 << 26, E=1024, K=65536, N=65536, fmt="bf16"), dict(call="linear", rows=1 << 26, K=8, N=65536, fmt="f32"),
        dict(call="linear", rows=1 << 26, E=1024, K=8, N=8, fmt="bf16", how="odd")])
    for status, ls in calls:
        assert (status == 0) == bool(ls)
        assert all(threads < 1 << 32 for _, _, threads in ls)
