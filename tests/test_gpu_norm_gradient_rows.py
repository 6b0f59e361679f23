"""GPU: the gradient of the block norms where a workgroup walks several rows (more rows than
moe_block_norm_workspace has partial rows for) with several wavefronts, in each form of the kernel:
an input left out, up to eight wavefronts, up to sixteen.  Against the fp64 definition, and the same
bits on a second call."""
import numpy as np
import pytest
import torch

from test_gpu_block_norm import back, check_backward, grads, inputs
from test_gpu_tokens import B, F, R

pytestmark = pytest.mark.gpu


def check_rows(v, gate, h, y, dh=True, dx=True, only=None):
    """Gradients into two sets of buffers: right, and the same bits."""
    T, H = v["h"].shape
    assert R().moe_block_norm_workspace(T, H) < 2 * 4 * T * H    # fewer partial rows than rows
    first, again = grads(v, T, H, gate, only=only), grads(v, T, H, gate, only=only)
    for out in (first, again):
        back(v, v["h"], gate, 0.7, out, dh=dh, dx=dx)
    torch.cuda.synchronize()
    check_backward(v, v["h"], gate, 0.7, first, {"dh": h, "dy": y}, dh=dh, dx=dx)
    assert all(torch.equal(first[n], again[n]) for n in first)


WIDE = [(2000, 2048), (700, 4096), (600, 8192), (900, 8191), (3000, 1999), (2100, 513)]


@pytest.mark.parametrize("dh", [True, False])
@pytest.mark.parametrize("h,x", [(F, F), (B, B), (F, B)])
@pytest.mark.parametrize("T,H", WIDE)
def test_the_norm_alone(T, H, h, x, dh):
    """y = None: the gradient of a plain norm, from dx with and without dh_out."""
    v = dict(inputs(T, H, h, F, x, False, "none"), y=None)
    out = {n: torch.full_like(v[n], 9.0) for n in ("dh", "w_pre")}
    again = {n: torch.full_like(v[n], 9.0) for n in ("dh", "w_pre")}
    assert R().moe_block_norm_workspace(T, H) < 2 * 4 * T * H
    for o in (out, again):
        back(v, v["h"], "none", 1.0, {"dh": o["dh"], "dw_pre": o["w_pre"]}, dh=dh)
    torch.cuda.synchronize()
    check_backward(v, v["h"], "none", 1.0, {"dh": out["dh"], "dw_pre": out["w_pre"]}, {"dh": h}, dh=dh)
    assert all(torch.equal(out[n], again[n]) for n in out)


@pytest.mark.parametrize("gate,post", [("none", True), ("token", True), ("channel", False)])
@pytest.mark.parametrize("dh,dx", [(True, False), (False, True)])
@pytest.mark.parametrize("T,H", [(2000, 2048), (600, 8191)])
def test_one_gradient_comes_in(T, H, dh, dx, gate, post):
    v = inputs(T, H, B, F, B, post, gate)
    check_rows(v, gate, B, F, dh=dh, dx=dx, only=None if dx else ("dh", "dy", "dw_post", "dgate"))


@pytest.mark.parametrize("gate", ["none", "token", "channel"])
@pytest.mark.parametrize("h,y,x", [(B, B, B), (F, F, F), (B, F, B)])
@pytest.mark.parametrize("T,H", [(600, 8192), (700, 4104), (1100, 4095)])
def test_every_input(T, H, h, y, x, gate):
    """Sixteen wavefronts, and eight with the next row loaded ahead."""
    check_rows(inputs(T, H, h, y, x, True, gate), gate, h, y)


def test_the_norm_alone_in_place_and_captured():
    """dh in dh_out's place, and a captured pass replayed on new inputs with eager work between."""
    T, H = 1500, 2048
    v = dict(inputs(T, H, F, F, B, False, "none"), y=None)
    ws = torch.empty(R().moe_block_norm_workspace(T, H), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty_like(ws)
    dh, dw = torch.empty_like(v["h"]), torch.empty_like(v["w_pre"])
    want, wdw = torch.empty_like(dh), torch.empty_like(dw)

    def run(ws, dh, dw, dh_out=None):
        w = v if dh_out is None else dict(v, dh=dh_out)
        back(w, v["h"], "none", 1.0, {"dh": dh, "dw_pre": dw}, ws=ws)

    run(ws, want, wdw)
    same = v["dh"].clone()
    run(ws, same, dw, dh_out=same)
    torch.cuda.synchronize()
    assert torch.equal(same, want) and torch.equal(dw, wdw)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            run(ws, dh, dw)
    for _ in range(3):
        v["h"].normal_()
        v["dx"].normal_()
        torch.cuda.synchronize()
        g.replay()
        run(ws2, want, wdw)
        torch.cuda.synchronize()
        assert torch.equal(dh, want) and torch.equal(dw, wdw)
