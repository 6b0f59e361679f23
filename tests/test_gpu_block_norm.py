"""GPU: the norms around a block and their gradient against the fp64 definitions, and the whole frame
around the experts run together (a decode step through every layer, a training step)."""
import itertools

import numpy as np
import pytest
import torch

from oracle import norm, tokens
from test_gpu_tokens import B, F, R, U32, around, dev, f64, routing, views, within

pytestmark = pytest.mark.gpu

EPS = 1e-6
GATES = ("none", "token", "channel")


def depth(H):
    """Additions a term of a row's sum passes through: 8 in its thread, six between lanes, up to
    sixteen between wavefronts."""
    return 8 + 6 + 16


def kind(gate):
    r = R()
    return {"none": r.MOE_GATE_NONE, "token": r.MOE_GATE_TOKEN, "channel": r.MOE_GATE_CHANNEL}[gate]


def inputs(T, H, h, y, x, post, gate, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * T + H)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    v = {"h": (2 * rn(T, H)).to(h), "y": (0.5 * rn(T, H)).to(y), "w_pre": 1 + 0.3 * rn(H),
         "w_post": 1 + 0.3 * rn(H) if post else None,
         "gate": None if gate == "none" else rn(T if gate == "token" else H), "dh": rn(T, H).to(h), "dx": rn(T, H).to(x)}
    if T > 2:
        v["y"][1] = 0                 # a row whose rms is eps alone
        v["h"][2] = 0
        v["y"][2] = 0                 # and a residual row of zeros
    return v


def n64(t):
    return None if t is None else f64(t)


def check_forward(v, gate, alpha, h_out, x_out, h_type, x_type):
    H = v["h"].shape[1]
    rh, rx = norm.block_norm(f64(v["h"]), f64(v["y"]), n64(v["w_post"]), n64(v["gate"]), gate == "token",
                             n64(v["w_pre"]), alpha, EPS)
    add = np.abs(rh - f64(v["h"]))
    rho = (depth(H) / 2 + 6) * U32                         # of 1 / rms: the sum under a root, then three roundings
    eh = add * (rho + 6 * U32) + U32 * np.abs(rh)
    within(h_out, rh, eh, h_type)
    if x_out is None:
        return
    rms = np.sqrt(np.mean(rh * rh, 1, keepdims=True) + EPS)
    er = np.sqrt(np.mean(eh * eh, 1, keepdims=True)) / rms + rho
    within(x_out, rx, np.abs(f64(v["w_pre"])) / rms * eh + np.abs(rx) * (er + 4 * U32), x_type)


def check_backward(v, h_out, gate, alpha, got, types, dh=True, dx=True):
    H = h_out.shape[1]
    ref = norm.block_norm_backward(f64(h_out), n64(v["y"]), n64(v["w_post"]), n64(v["gate"]), gate == "token",
                                   n64(v["w_pre"]) if dx else None, f64(v["dh"]) if dh else None,
                                   f64(v["dx"]) if dx else None, alpha, EPS, depth(H), U32)
    for name, t in got.items():
        within(t, ref[name][0], ref[name][1], types.get(name, F))


def grads(v, T, H, gate, fill=9.0, only=None):
    out = {"dh": torch.full_like(v["dh"], fill), "dy": torch.full_like(v["y"], fill), "dw_pre": torch.full_like(v["w_pre"], fill)}
    if v["w_post"] is not None:
        out["dw_post"] = torch.full_like(v["w_post"], fill)
    if gate != "none":
        out["dgate"] = torch.full_like(v["gate"], fill)
    return out if only is None else {n: t for n, t in out.items() if n in only}


def back(v, h_out, gate, alpha, out, dh=True, dx=True, ws=True, stream=None):
    r = R()
    T, H = h_out.shape
    w = torch.empty(r.moe_block_norm_workspace(T, H), dtype=torch.uint8, device="cuda") if ws is True else ws
    r.moe_block_norm_backward(h_out, v["y"], v["w_post"], v["gate"], v["w_pre"] if dx else None, v["dh"] if dh else None,
                              v["dx"] if dx else None, out.get("dh"), out.get("dy"), out.get("dw_post"), out.get("dgate"),
                              out.get("dw_pre"), w, gate_kind=kind(gate), alpha=alpha, eps=EPS, stream=stream)


SHAPES = [(1, 1), (1, 2048), (2, 7), (3, 64), (5, 513), (4, 4096), (33, 1999), (9, 8192), (3, 8191), (2, 4104), (700, 96),
          (300, 2056)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("h,y,x", itertools.product((F, B), repeat=3))
def test_block_norm_and_gradient(T, H, h, y, x):
    """Every type, with the gate and the post-norm turning over the shapes."""
    n = SHAPES.index((T, H)) + (h is B) + 2 * (y is B)
    gate, post, alpha = GATES[n % 3], n % 4 != 3, (1.0, 0.37)[n % 2]
    v = inputs(T, H, h, y, x, post, gate)
    for how in ("dense", "gaps", "odd"):
        w = dict(v, h=views(v["h"], how), y=views(v["y"], how))
        h_out = views(torch.full((T, H), 9.0, dtype=h, device="cuda"), how)
        x_out = views(torch.full((T, H), 9.0, dtype=x, device="cuda"), how)
        R().moe_block_norm(w["h"], w["y"], v["w_post"], v["gate"], v["w_pre"], h_out, x_out, gate_kind=kind(gate), alpha=alpha,
                           eps=EPS)
        check_forward(v, gate, alpha, h_out, x_out, h, x)
        assert (around(h_out) == 55.0).all() and (around(x_out) == 55.0).all()
        if how == "dense":
            same = v["h"].clone()
            R().moe_block_norm(same, v["y"], v["w_post"], v["gate"], v["w_pre"], same, x_out, gate_kind=kind(gate), alpha=alpha,
                               eps=EPS)
            assert torch.equal(same, h_out)                       # in place
            keep = h_out
    out = grads(v, T, H, gate)
    back(v, keep, gate, alpha, out)
    check_backward(v, keep, gate, alpha, out, {"dh": h, "dy": y})
    again = grads(v, T, H, gate)
    back(v, keep, gate, alpha, again)
    assert all(torch.equal(out[n], again[n]) for n in out)        # the same bits every time
    if T > 1:                                                     # rows with gaps, and off 16 bytes
        for how in ("gaps", "odd"):
            w = {n: views(t, how) if n in ("y", "dh", "dx") else t for n, t in v.items()}
            o = {n: views(t, how) if n in ("dh", "dy") else t for n, t in grads(v, T, H, gate).items()}
            back(w, views(keep, how), gate, alpha, o)
            assert all(torch.equal(out[n], o[n]) for n in out)
            assert (around(o["dh"]) == 55.0).all() and (around(o["dy"]) == 55.0).all()


@pytest.mark.parametrize("gate,post", itertools.product(GATES, (True, False)))
def test_parts(gate, post):
    """Each input and output that may be left out, and gradients in their inputs' places."""
    T, H, alpha = 70, 520, 0.8
    r = R()
    v = inputs(T, H, B, F, B, post, gate)
    h_out = torch.empty_like(v["h"])
    r.moe_block_norm(v["h"], v["y"], v["w_post"], v["gate"], None, h_out, None, gate_kind=kind(gate), alpha=alpha, eps=EPS)
    check_forward(v, gate, alpha, h_out, None, B, B)
    if gate == "none" and not post:                               # the second norm alone
        x_out = torch.empty_like(v["dx"])
        r.moe_block_norm(v["h"], None, None, None, v["w_pre"], None, x_out, eps=EPS)
        rh, rx = norm.block_norm(f64(v["h"]), None, None, None, False, f64(v["w_pre"]), 1.0, EPS)
        within(x_out, rx, np.abs(rx) * (depth(H) + 8) * U32, B)
        dh, dwp = torch.empty_like(v["h"]), torch.empty_like(v["w_pre"])
        w = dict(v, y=None, w_post=None, gate=None)
        for with_dh in (True, False):
            o = {"dh": dh, "dw_pre": dwp}
            back(w, v["h"], gate, 1.0, o, dh=with_dh)
            check_backward(w, v["h"], gate, 1.0, o, {"dh": B}, dh=with_dh)
    full = grads(v, T, H, gate)
    back(v, h_out, gate, alpha, full)
    types = {"dh": B, "dy": F}
    for names in (("dh",), ("dy",), ("dw_pre",), ("dw_post",), ("dgate",), ("dh", "dy"), ("dw_post", "dgate")):
        o = grads(v, T, H, gate, only=names)
        if o:
            back(v, h_out, gate, alpha, o, ws=None if set(o) <= {"dh", "dy"} else True)
            assert all(torch.equal(o[n], full[n]) for n in o if n in ("dh", "dy"))
            check_backward(v, h_out, gate, alpha, o, types)
    for with_dh, with_dx in ((False, True), (True, False)):
        o = grads(v, T, H, gate, only=None if with_dx else ("dh", "dy", "dw_post", "dgate"))
        back(v, h_out, gate, alpha, o, dh=with_dh, dx=with_dx)
        check_backward(v, h_out, gate, alpha, o, types, dh=with_dh, dx=with_dx)
    w = dict(v, y=v["y"].clone(), dh=v["dh"].clone())
    o = dict(grads(v, T, H, gate), dh=w["dh"], dy=w["y"])
    back(w, h_out, gate, alpha, o)
    assert all(torch.equal(o[n], full[n]) for n in full)


def test_many_rows_of_weights_gradients():
    """Sums over more rows than there are workgroups, many times over."""
    T, H = 5000, 72
    v = inputs(T, H, F, B, B, True, "channel")
    h_out = v["h"]
    out = grads(v, T, H, "channel")
    back(v, h_out, "channel", 0.5, out)
    check_backward(v, h_out, "channel", 0.5, out, {"dh": F, "dy": B})


def test_infinities_stay_in_their_row():
    T, H = 4, 300
    v = inputs(T, H, F, F, F, True, "none")
    v["y"][0, 5] = float("inf")
    v["h"][3, 7] = float("nan")
    h_out, x_out = torch.empty_like(v["h"]), torch.empty_like(v["h"])
    R().moe_block_norm(v["h"], v["y"], v["w_post"], None, v["w_pre"], h_out, x_out, eps=EPS)
    assert h_out[0, 5].isnan() and x_out[0].isnan().all()         # inf / inf; the other channels add 0
    assert torch.equal(h_out[0, :5], v["h"][0, :5])
    assert h_out[3, 7].isnan() and x_out[3].isnan().all() and not h_out[3, :7].isnan().any()
    assert x_out[1:3].isfinite().all()


def test_offsets_past_32_bits():
    """Rows 2^31 elements into their buffers."""
    H = 8192
    T = (1 << 31) // H + 3
    y = torch.zeros(T, H, dtype=B, device="cuda")
    y[-1] = 1.0
    h = torch.zeros(T, H, dtype=B, device="cuda")
    x = torch.empty(T, H, dtype=B, device="cuda")
    w = torch.full((H,), 2.0, device="cuda")
    R().moe_block_norm(h, y, None, None, w, h, x, eps=EPS)
    assert (h[-1] == 1).all() and (x[-1] == 2).all() and not h[-2].any() and not x[-2].any()
    ws = torch.empty(R().moe_block_norm_workspace(T, H), dtype=torch.uint8, device="cuda")
    dwp = torch.empty(H, device="cuda")
    R().moe_block_norm_backward(h, y, None, None, w, x, x, None, y, None, None, dwp, ws, eps=EPS)
    # dx = 2 on the last row alone, where h' / rms is 1 up to eps / 2
    assert (dwp - 2.0).abs().max() <= 2.0 * (EPS + 64 * U32)
    # d = 4 in every channel: d - h' mean(d h') / rms^2 is about 4 eps, so dy = dh = 2 to bf16
    assert ((y[-1].float() - 2).abs() <= 2 * 2.0 ** -8).all() and not y[-2].any()


def test_streams_and_graph_replays():
    r = R()
    T, H = 300, 1024
    v = inputs(T, H, B, B, B, True, "channel")
    h_out, x_out = torch.empty_like(v["h"]), torch.empty_like(v["dx"])
    outs = [grads(v, T, H, "channel") for _ in range(3)]
    wss = [torch.empty(r.moe_block_norm_workspace(T, H), dtype=torch.uint8, device="cuda") for _ in range(3)]

    def forward():
        r.moe_block_norm(v["h"], v["y"], v["w_post"], v["gate"], v["w_pre"], h_out, x_out, gate_kind=r.MOE_GATE_CHANNEL, eps=EPS)

    forward()
    back(v, h_out, "channel", 1.0, outs[0], ws=wss[0])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        back(v, h_out, "channel", 1.0, outs[1], ws=wss[1], stream=s1)
        back(v, h_out, "channel", 1.0, outs[2], ws=wss[2], stream=s2)
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert all(torch.equal(o[n], outs[0][n]) for n in o)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            forward()
            back(v, h_out, "channel", 1.0, outs[1], ws=wss[1])
    for i in range(3):
        v["h"].normal_()
        v["dx"].normal_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [h_out.clone(), x_out.clone()] + [t.clone() for t in outs[1].values()]
        forward()
        back(v, h_out, "channel", 1.0, outs[1], ws=wss[0])
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, [h_out, x_out] + list(outs[1].values())))


# --- the frame as it is used -------------------------------------------------
@pytest.mark.parametrize("mode", ["fused", "offload", "hybrid"])
@pytest.mark.parametrize("T", [1, 3])
def test_decode_block_is_its_two_steps(mode, T):
    """moe_decode_block over every layer, each layer's input the norm of the stream: the bits of
    moe_decode_layer and moe_block_norm, eagerly and from a captured graph."""
    import workloads as W
    from moe_harness import Harness
    r = R()
    wl = W.A3B_DECODE.with_(name="block", n_layers=3, n_experts=16, top_k=4, hidden=256, inter=128)
    m = {"fused": r.MOE_MODE_FUSED, "offload": r.MOE_MODE_OFFLOAD, "hybrid": r.MOE_MODE_HYBRID}[mode]
    n_slots = 8 if mode == "hybrid" else 32
    ctxs = [Harness(wl, m, n_slots=n_slots, bw=(25_000_000_000, 100_000_000_000), flags=r.MOE_FLAG_DEVICE_FILLS)
            for _ in range(2)]
    H, k, Ln = wl.hidden, wl.top_k, wl.n_layers
    g = torch.Generator(device="cuda").manual_seed(3)
    w_post, w_pre = (1 + 0.2 * torch.randn(Ln, H, device="cuda", generator=g) for _ in range(2))
    gate = torch.rand(H, device="cuda", generator=g)
    cfg = r.moe_norm_config(T, H, F_FMT(r, F), F_FMT(r, F), F_FMT(r, B), r.MOE_GATE_CHANNEL, 0.5, EPS, 0, 0, 0)

    class Bufs:
        def __init__(self):
            self.h = torch.empty(T, H, device="cuda")
            self.x = torch.empty(T, H, dtype=B, device="cuda")
            self.y = torch.empty(Ln, T, H, device="cuda")
            self.idx = torch.empty(Ln, T, k, dtype=torch.int32, device="cuda")
            self.slot = torch.empty(Ln, T, k, dtype=torch.int32, device="cuda")
            self.w = torch.empty(Ln, T, k, device="cuda")

        def outputs(self):
            return [t.clone() for t in (self.h, self.x, self.y, self.idx, self.slot, self.w)]

    a, b = Bufs(), Bufs()

    def fused_step(ctx, u):
        r.moe_block_norm(u.h, None, None, None, w_pre[0], None, u.x, eps=EPS)
        for l in range(Ln):
            last = l == Ln - 1
            r.moe_decode_block(ctx, l, u.x, T, None, u.idx[l], u.w[l], u.slot[l], u.y[l], cfg, u.h, w_post[l], gate,
                               None if last else w_pre[l + 1], None if last else u.x)

    def two_steps(ctx, u):
        r.moe_block_norm(u.h, None, None, None, w_pre[0], None, u.x, eps=EPS)
        for l in range(Ln):
            last = l == Ln - 1
            r.moe_decode_layer(ctx, l, u.x, T, None, u.idx[l], u.w[l], u.slot[l], u.y[l])
            r.moe_block_norm(u.h, u.y[l], w_post[l], gate, None if last else w_pre[l + 1], u.h, None if last else u.x,
                             gate_kind=r.MOE_GATE_CHANNEL, alpha=0.5, eps=EPS)

    for step in range(3):
        h0 = torch.randn(T, H, device="cuda", generator=g)
        a.h.copy_(h0)
        b.h.copy_(h0)
        fused_step(ctxs[0].ctx, a)
        two_steps(ctxs[1].ctx, b)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a.outputs(), b.outputs())), step
        assert a.h.isfinite().all() and not torch.equal(a.h, h0)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            fused_step(ctxs[0].ctx, a)
    for step in range(4):
        h0 = torch.randn(T, H, device="cuda", generator=g)
        a.h.copy_(h0)
        b.h.copy_(h0)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            gr.replay()
        r.moe_sync(ctxs[0].ctx, s)
        two_steps(ctxs[1].ctx, b)
        torch.cuda.synchronize()
        got, want = a.outputs(), b.outputs()
        assert torch.equal(got[3], want[3]) and torch.equal(got[4], want[4])
        assert all(torch.equal(p, q) for p, q in zip(got, want)), step


def F_FMT(r, dtype):
    return r.MOE_AFMT_BF16 if dtype is B else r.MOE_AFMT_F32


def test_decode_block_refuses():
    import workloads as W
    from moe_harness import Harness
    r = R()
    h = Harness(W.TINY, r.MOE_MODE_OFFLOAD, n_slots=4)
    H, k = W.TINY.hidden, W.TINY.top_k
    x, y, hs = (torch.zeros(1, H, device="cuda") for _ in range(3))
    idx, slot = (torch.zeros(1, k, dtype=torch.int32, device="cuda") for _ in range(2))
    w, wp = torch.zeros(1, k, device="cuda"), torch.ones(H, device="cuda")
    good = dict(T=1, H=H, h=0, y=0, x=0, gate=0, alpha=1.0, eps=EPS, lh=0, ly=0, lx=0)
    before = h.snapshot()
    for bad in (dict(T=2), dict(H=H // 2), dict(y=1), dict(ly=H + 8), dict(eps=0.0), dict(gate=1)):
        cfg = r.moe_norm_config(*{**good, **bad}.values())
        with pytest.raises(r.MoeError) as e:
            r.moe_decode_block(h.ctx, 0, x, 1, None, idx, w, slot, y, cfg, hs, None, None, wp, x)
        assert e.value.status == r.MOE_EINVAL
    with pytest.raises(r.MoeError):
        r.moe_decode_block(h.ctx, 0, x, 1, None, idx, w, slot, y, r.moe_norm_config(*good.values()), y, None, None, wp, x)
    torch.cuda.synchronize()
    assert all(np.array_equal(p, q) for p, q in zip(before, h.snapshot()))      # nothing ran


def test_training_step_through_the_frame():
    """stream -> norm -> router -> sort and move -> experts -> weighted return -> gated residual -> norm, and
    all the way back, against autograd in fp64.  The stages run in fp32, each a few roundings of sums of at
    most 64 terms, so every gradient agrees to 1e-4 of its largest element."""
    import workloads as W
    from moe_harness import Harness
    r = R()
    T, H, E, k, I, alpha, eps = 40, 64, 8, 2, 32, 0.6, 1e-5
    wl = W.TINY.with_(n_experts=E, top_k=k, hidden=H, renorm=1)
    h = Harness(wl, r.MOE_MODE_OFFLOAD, n_slots=1, max_tokens=T)
    g = torch.Generator(device="cuda").manual_seed(5)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    h0, wr = rn(T, H), rn(E, H) / H ** 0.5
    w_in, w_post, w_pre, gate = 1 + 0.1 * rn(H), 1 + 0.1 * rn(H), 1 + 0.1 * rn(H), torch.rand(T, device="cuda", generator=g)
    w1, w2 = rn(E, I, H) / H ** 0.5, rn(E, H, I) / I ** 0.5
    dh_out, dx_out = rn(T, H), rn(T, H)
    new = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    ints = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731

    x = new(T, H)
    r.moe_block_norm(h0, None, None, None, w_in, None, x, eps=eps)
    z = x @ wr.t()
    idx, gates = ints(T, k), new(T, k)
    r.moe_topk(h.ctx, z, T, idx, gates)
    xs, perm, inv, off = new(T * k, H), ints(T * k), ints(T, k), ints(E + 1)
    ws = torch.empty(r.moe_dispatch_workspace(T, k, E), dtype=torch.uint8, device="cuda")
    r.moe_dispatch(idx, E, x, xs, perm, inv, off, ws)
    bounds = off.tolist()
    ys = new(T * k, H)
    for e in range(E):
        rows = slice(bounds[e], bounds[e + 1])
        ys[rows] = torch.relu(xs[rows] @ w1[e].t()) @ w2[e].t()
    y, h1, x1 = new(T, H), new(T, H), new(T, H)
    r.moe_combine(ys, inv, gates, y)
    r.moe_block_norm(h0, y, w_post, gate, w_pre, h1, x1, gate_kind=r.MOE_GATE_TOKEN, alpha=alpha, eps=eps)
    # back
    nw = torch.empty(r.moe_block_norm_workspace(T, H), dtype=torch.uint8, device="cuda")
    dh, dy, dwq, dwp, dg = new(T, H), new(T, H), new(H), new(H), new(T)
    r.moe_block_norm_backward(h1, y, w_post, gate, w_pre, dh_out, dx_out, dh, dy, dwq, dg, dwp, nw,
                              gate_kind=r.MOE_GATE_TOKEN, alpha=alpha, eps=eps)
    dys, dgates = new(T * k, H), new(T, k)
    r.moe_combine_backward(dy, ys, inv, gates, dys, dgates)
    dxs, dw1, dw2 = new(T * k, H), torch.zeros_like(w1), torch.zeros_like(w2)
    for e in range(E):
        rows = slice(bounds[e], bounds[e + 1])
        pre = xs[rows] @ w1[e].t()
        dw2[e] = dys[rows].t() @ torch.relu(pre)
        da = (dys[rows] @ w2[e]) * (pre > 0)
        dw1[e] = da.t() @ xs[rows]
        dxs[rows] = da @ w1[e]
    dx, dz = new(T, H), new(T, E)
    r.moe_dispatch_backward(dxs, inv, dx)
    r.moe_topk_backward(z, idx, dgates, 1, dz)
    dx += dz @ wr
    dwr = dz.t() @ x
    dh0, dwin = new(T, H), new(H)
    r.moe_block_norm_backward(h0, None, None, None, w_in, dh, dx, dh0, None, None, None, dwin, nw, eps=eps)
    torch.cuda.synchronize()

    leaf = {n: t.double().cpu().requires_grad_() for n, t in
            dict(h0=h0, wr=wr, w_in=w_in, w_post=w_post, w_pre=w_pre, gate=gate, w1=w1, w2=w2).items()}
    rms = lambda v: v / (v.pow(2).mean(1, keepdim=True) + eps).sqrt()  # noqa: E731
    X = leaf["w_in"] * rms(leaf["h0"])
    Z = X @ leaf["wr"].t()
    at = idx.cpu().long()
    G = torch.softmax(Z.gather(1, at), 1)
    Y = torch.zeros(T, H, dtype=torch.float64)
    for j in range(k):
        a = torch.relu(torch.matmul(leaf["w1"][at[:, j]], X[:, :, None]))
        Y = Y + G[:, j, None] * torch.matmul(leaf["w2"][at[:, j]], a)[:, :, 0]
    H1 = leaf["h0"] + alpha * leaf["gate"][:, None] * leaf["w_post"] * rms(Y)
    X1 = leaf["w_pre"] * rms(H1)
    ((H1 * dh_out.double().cpu()).sum() + (X1 * dx_out.double().cpu()).sum()).backward()
    for got, want in ((h1, H1), (x1, X1), (y, Y)):
        assert np.abs(f64(got) - want.detach().numpy()).max() <= 1e-5 * want.detach().abs().max()
    for name, got in dict(h0=dh0, wr=dwr, w_in=dwin, w_post=dwq, w_pre=dwp, gate=dg, w1=dw1, w2=dw2).items():
        ref = leaf[name].grad.numpy()
        assert np.abs(f64(got) - ref).max() <= 1e-4 * np.abs(ref).max(), name
