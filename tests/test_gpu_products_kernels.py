"""GPU: every kernel of the experts' products against the fp64 definitions, at sizes that test_products_kernels.py holds to
their kernels, with all that an epilogue can do, rows that no expert has and uneven experts."""
import pytest
import torch

from oracle import products
from product_sizes import SIZES, case
from test_gpu_products import B, F, UOUT, R, Out, act_kind, dev, f64, fmt_of, layout, operands, poison, uneven

pytestmark = pytest.mark.gpu

DT = {"bf16": B, "f32": F}


def name(row):
    c, kernel = case(row)
    return f"{c['call']}-{c['rows']}-{c['E']}-{c['K']}-{c['N']}-{c['fmt']}-{kernel[0]}"


@pytest.mark.parametrize("row", SIZES, ids=name)
def test_kernel(row):
    c, _ = case(row)
    L, rows, E, K, N, how, act, dtype = R(), c["rows"], max(c["E"], 1), c["K"], c["N"], c["how"], c["act"], DT[c["fmt"]]
    glu, off = c["call"].startswith("glu"), uneven(rows, c["E"], min(rows // 10, 40)) if c["E"] else None
    cols = 2 * N if glu else N
    x, w, rnd = operands(rows, E, K, cols, dtype, how)
    if not c["call"].endswith("backward"):
        poisoned = poison(x.clone() if how == "dense" else layout(x.clone(), how), off, rows)
        if glu:
            ref, kept = products.glu(f64(x), f64(w), off, act)
            out, saved = Out(dtype, how, rows, N), Out(dtype, how, rows, cols)
            L.moe_glu(poisoned, w, out.t, saved.t, dev(off), act=act_kind(act))
            names = ("a", "gu")
        else:
            bias, r = rnd(E, N), layout(rnd(rows, N).to(dtype), how)
            ref, kept = products.linear(f64(x), f64(w), f64(bias), f64(r), off, act)
            out, saved = Out(dtype, how, rows, N), Out(dtype, how, rows, N)
            L.moe_linear(poisoned, w, out.t, bias, r, saved.t, dev(off), act=act_kind(act))
            names = ("y", "z")
        out.check(names[0], ref[names[0]], kept)
        saved.check(names[1], ref[names[1]], kept)
        return
    dy, z = layout(rnd(rows, N).to(dtype), how), layout(rnd(rows, cols).to(dtype), how)
    outs = {"dx": Out(dtype, how, rows, K), "dw": Out(dtype, "dense", E, cols, K), "dbias": Out(F, "dense", E, N)}
    outs = {n: o for n, o in outs.items() if n in c["out"]}
    t = {n: o.t for n, o in outs.items()}
    size = (L.moe_glu_workspace if glu else L.moe_linear_workspace)(rows, E, K, N, fmt_of(dtype))
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    if glu:
        ref, kept = products.glu_backward(f64(dy), f64(z), f64(x), f64(w), off, act, UOUT[dtype])
    else:
        ref, kept = products.linear_backward(f64(dy), f64(z), f64(x), f64(w), off, act, UOUT[dtype] if act != "none" else 0.0)
    for v in (x, dy, z):
        poison(v, off, rows)
    if glu:
        L.moe_glu_backward(dy, z, x, w, t.get("dx"), t.get("dw"), ws, dev(off), act=act_kind(act))
    else:
        L.moe_linear_backward(dy, z if act != "none" else None, x, w, t.get("dx"), t.get("dw"), t.get("dbias"), ws, dev(off), act=act_kind(act))
    for n, o in outs.items():
        o.check(n, ref[n], kept if n == "dx" else None)
