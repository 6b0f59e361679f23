"""GPU: moe_block_norm without a block's output (the first norm of a chain) and its gradient, over row
lengths, types and layouts, against the fp64 definitions."""
import itertools

import numpy as np
import pytest
import torch

from oracle import norm
from test_gpu_block_norm import EPS, back, check_backward, depth, inputs
from test_gpu_tokens import B, F, R, U32, around, f64, views, within

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 2048), (3, 7), (2, 8), (5, 513), (33, 1999), (9, 8191), (4, 8192), (300, 2056), (4000, 64)]


@pytest.mark.parametrize("how", ["dense", "gaps", "odd"])
@pytest.mark.parametrize("h,x", itertools.product((F, B), repeat=2))
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm_alone(T, H, h, x, how):
    v = inputs(T, H, h, F, x, False, "none")
    x_out = views(torch.full((T, H), 9.0, dtype=x, device="cuda"), how)
    R().moe_block_norm(views(v["h"], how), None, None, None, v["w_pre"], None, x_out, eps=EPS)
    rx = norm.block_norm(f64(v["h"]), None, None, None, False, f64(v["w_pre"]), 1.0, EPS)[1]
    within(x_out, rx, np.abs(rx) * (depth(H) + 8) * U32, x)
    assert (around(x_out) == 55.0).all()


@pytest.mark.parametrize("how", ["dense", "gaps", "odd"])
@pytest.mark.parametrize("h,x", itertools.product((F, B), repeat=2))
@pytest.mark.parametrize("T,H", SHAPES)
def test_gradient_alone(T, H, h, x, how):
    v = dict(inputs(T, H, h, F, x, False, "none"), y=None)
    w = dict(v, dh=views(v["dh"], how), dx=views(v["dx"], how))
    hv = views(v["h"], how)
    for dh in (True, False):
        both = {"dh": views(torch.full_like(v["dh"], 9.0), how), "dw_pre": torch.full_like(v["w_pre"], 9.0)}
        back(w, hv, "none", 1.0, both, dh=dh)
        check_backward(v, v["h"], "none", 1.0, both, {"dh": h}, dh=dh)
        assert (around(both["dh"]) == 55.0).all()
        for name in both:                                  # either output alone: the same bits of dh
            one = {name: both[name].clone() if name == "dw_pre" else views(torch.full_like(v["dh"], 9.0), how)}
            back(w, hv, "none", 1.0, one, dh=dh, ws=None if name == "dh" else True)
            check_backward(v, v["h"], "none", 1.0, one, {"dh": h}, dh=dh)
            assert name != "dh" or torch.equal(one["dh"], both["dh"])
    same = views(v["dh"].clone(), how)
    back(dict(w, dh=same), hv, "none", 1.0, {"dh": same}, ws=None)     # in dh_out's place
    want = views(torch.full_like(v["dh"], 9.0), how)
    back(w, hv, "none", 1.0, {"dh": want}, ws=None)
    assert torch.equal(same, want) and (around(same) == 55.0).all()


def test_gradient_alone_against_differences():
    """sum(dx * norm(h)) along a direction: the fp64 forward's central difference against <dh, way>."""
    T, H, step = 6, 200, 2.0 ** -12
    v = inputs(T, H, F, F, F, False, "none")
    v["h"][2] = 1.0                        # rows of zeros are as steep as 1 / eps: not here
    dh, dw = torch.empty_like(v["h"]), torch.empty_like(v["w_pre"])
    back(dict(v, y=None), v["h"], "none", 1.0, {"dh": dh, "dw_pre": dw}, dh=False)
    h, w, dx = f64(v["h"]), f64(v["w_pre"]), f64(v["dx"])
    rng = np.random.default_rng(0)
    wh, ww = rng.standard_normal(h.shape), rng.standard_normal(w.shape)
    f = lambda s: np.sum(dx * norm.block_norm(h + s * wh, None, None, None, False, w + s * ww, 1.0, EPS)[1], axis=1)  # noqa: E731
    num = np.sum(f(step) - f(-step)) / (2 * step)
    ana = np.sum(f64(dh) * wh) + np.sum(f64(dw) * ww)
    # third derivatives along a direction of size |wh| / rms(h) are at most about 10 (|wh| / rms)^3 of the sum
    # of magnitudes, with rms(h) >= 1 here; the gradients err by (depth + T + 50) U32 of theirs
    size = np.sum(np.abs(dx * w) * (1 + np.abs(wh) + np.abs(h))) + np.sum(np.abs(dx * h * ww[None]))
    assert abs(num - ana) <= size * (10 * step ** 2 + (depth(H) + T + 50) * U32)
