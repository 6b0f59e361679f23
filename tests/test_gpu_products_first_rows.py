"""GPU: tables of experts that begin above the first row: rows before the first expert's are no expert's, as those
behind the last one's are, so nothing of them is read or written."""
import numpy as np
import pytest
import torch

from oracle import products
from test_gpu_products import B, F, FILL, UOUT, R, Out, act_kind, dev, each, f64, fmt_of, layout, operands, types

pytestmark = pytest.mark.gpu


def table(first, sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32) + np.int32(first)


def poison(off, *ts):
    for t in ts:
        if t is not None:
            t[:int(off[0])] = float("nan")
            t[int(off[-1]):] = float("nan")


# rows, the first expert's first row, experts' sizes, K (H), N (I): short and long sums; a k cut across workgroups (dx
# of few rows, dw of small weights); sizes of one launch for both gradients and of one each
TABLES = [(40, 7, [0, 20, 3], 72, 40), (300, 130, [100, 0, 40], 136, 72), (9, 8, [1], 64, 64), (50, 50, [0, 0], 64, 64), (20, 3, [5, 9], 24, 4000),
          (2500, 300, [2100], 72, 64), (3000, 17, [1400, 1500], 65, 99), (1100, 64, [300, 600, 100], 640, 512)]


@types
@pytest.mark.parametrize("rows,first,sizes,K,N", TABLES)
def test_rows_before_the_first_expert(dtype, rows, first, sizes, K, N):
    L, E, off = R(), len(sizes), table(first, sizes)
    u = UOUT[dtype]
    x, w, rnd = operands(rows, E, K, 2 * N, dtype, "dense")
    gu, da = rnd(rows, 2 * N).to(dtype), rnd(rows, N).to(dtype)
    clean = [f64(t) for t in (x, gu, da)]
    poison(off, x, gu, da)
    ref, kept = products.glu(clean[0], f64(w), off, "silu")
    a, g = Out(dtype, "dense", rows, N), Out(dtype, "dense", rows, 2 * N)
    L.moe_glu(x, w, a.t, g.t, dev(off))
    a.check("a", ref["a"], kept)
    g.check("gu", ref["gu"], kept)
    ref, kept = products.glu_backward(clean[2], clean[1], clean[0], f64(w), off, "silu", u)
    dx, dw = Out(dtype, "dense", rows, K), Out(dtype, "dense", E, 2 * N, K)
    ws = torch.full((L.moe_glu_workspace(rows, E, K, N, fmt_of(dtype)),), 255, dtype=torch.uint8, device="cuda")
    L.moe_glu_backward(da, gu, x, w, dx.t, dw.t, ws, dev(off))
    dx.check("dx", ref["dx"], kept)
    dw.check("dw", ref["dw"])

    w2 = w[:, :N].contiguous()
    dy, z, bias = rnd(rows, N).to(dtype), rnd(rows, N).to(dtype), rnd(E, N)
    clean = clean[:1] + [f64(dy), f64(z)]
    poison(off, dy, z)
    ref, kept = products.linear(clean[0], f64(w2), f64(bias), None, off, "gelu")
    y = Out(dtype, "dense", rows, N)
    L.moe_linear(x, w2, y.t, bias, offsets=dev(off), act=act_kind("gelu"))
    y.check("y", ref["y"], kept)
    ws = torch.full((L.moe_linear_workspace(rows, E, K, N, fmt_of(dtype)),), 255, dtype=torch.uint8, device="cuda")
    for act, with_bias in (("gelu", True), ("gelu", False), ("none", True)):
        ref, kept = products.linear_backward(clean[1], clean[2], clean[0], f64(w2), off, act, u if act != "none" else 0.0)
        dx, dw, db = Out(dtype, "dense", rows, K), Out(dtype, "dense", E, N, K), Out(F, "dense", E, N)
        L.moe_linear_backward(dy, z, x, w2, dx.t, dw.t, db.t if with_bias else None, ws, dev(off), act=act_kind(act))
        dx.check("dx", ref["dx"], kept)
        dw.check("dw", ref["dw"])
        if with_bias:
            db.check("dbias", ref["dbias"])


@types
@pytest.mark.parametrize("call", ["glu", "linear"])
def test_the_gradient_before_the_products_begins_there_too(dtype, call):
    """The pass that forms dgu or dz (at the start of the workspace, a row of n elements rounded up to eight each) has
    nothing to do with rows before the first expert's or behind the last one's: their places keep what was there."""
    L, rows, first, sizes, K, N = R(), 700, 300, [64, 100], 72, 64
    E, off = len(sizes), table(300, sizes)
    n = 2 * N if call == "glu" else N
    x, w, rnd = operands(rows, E, K, n, dtype, "dense")
    z, dy = rnd(rows, n).to(dtype), rnd(rows, N).to(dtype)
    size = (L.moe_glu_workspace if call == "glu" else L.moe_linear_workspace)(rows, E, K, N, fmt_of(dtype))
    ws = torch.full((size,), 171, dtype=torch.uint8, device="cuda")
    assert ws.data_ptr() % 16 == 0
    dx, dw = torch.empty(rows, K, dtype=dtype, device="cuda"), torch.empty_like(w)
    if call == "glu":
        L.moe_glu_backward(dy, z, x, w, dx, dw, ws, dev(off))
    else:
        L.moe_linear_backward(dy, z, x, w, dx, dw, None, ws, dev(off), act=L.MOE_ACT_SILU)
    d = ws[:rows * n * dtype.itemsize].view(rows, -1)
    last = int(off[-1])
    assert (d[:first] == 171).all() and (d[last:] == 171).all() and not (d[first:last] == 171).all(1).any()
