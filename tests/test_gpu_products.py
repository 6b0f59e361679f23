"""GPU: the experts' products and their gradients against the fp64 definitions, within bounds derived per
element (oracle/products.py) and the output's own rounding: 2^-8 of the value for bf16, 2^-24 for fp32."""
import numpy as np
import pytest
import torch

from oracle import products

pytestmark = pytest.mark.gpu

F, B = torch.float32, torch.bfloat16
UOUT = {F: 2.0 ** -24, B: 2.0 ** -8}
FILL = 55.0


def R():
    import routed_expert_ffn_02_amd
    return routed_expert_ffn_02_amd


def act_kind(act):
    return {"none": R().MOE_ACT_NONE, "silu": R().MOE_ACT_SILU, "gelu": R().MOE_ACT_GELU}[act]


def fmt_of(dtype):
    return R().MOE_AFMT_BF16 if dtype == B else R().MOE_AFMT_F32


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def within(name, got, ref, dtype):
    value, err = ref
    got = f64(got).reshape(value.shape)
    tol = err + UOUT[dtype] * (np.abs(value) + err) + 1e-37
    bad = ~(np.abs(got - value) <= tol)
    assert not bad.any(), (name, int(bad.sum()), float((np.abs(got - value) / tol).max()), np.argwhere(bad)[:4].tolist())


def layout(t, how):
    """The values of t [.., n] in a layout: dense; rows with gaps that keep 16 bytes; starting one element off."""
    if how == "dense":
        return t.contiguous()
    pad, first = (24, 8) if how == "gaps" else (3, 1)
    buf = torch.full((*t.shape[:-1], t.shape[-1] + pad), FILL, dtype=t.dtype, device="cuda")
    buf[..., first:first + t.shape[-1]] = t
    return buf[..., first:first + t.shape[-1]]


class Out:
    """An output filled with FILL, in a layout, whose surroundings must stay."""

    def __init__(self, dtype, how, *shape):
        self.t = layout(torch.full(shape, FILL, dtype=dtype, device="cuda"), how)
        self.dtype = dtype

    def check(self, name, ref, kept=None):
        got = self.t
        if kept is not None:
            k = torch.from_numpy(kept).cuda()
            assert (got[~k] == FILL).all(), name                 # rows without an expert
            within(name, got[k], (ref[0][kept], ref[1][kept]), self.dtype)
        else:
            within(name, got, ref, self.dtype)
        if self.t._base is not None:
            base = self.t._base.clone()
            n = self.t.shape[-1]
            first = (self.t.storage_offset()) % base.shape[-1]
            base[..., first:first + n] = FILL
            assert (base == FILL).all(), name


def table(rows, sizes, tail=0):
    """offsets of these group sizes; the last `tail` rows have no expert."""
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    assert off[-1] == rows - tail
    return off


def uneven(rows, E, tail=0, seed=0):
    rng = np.random.default_rng(seed + 7 * rows + E)
    p = rng.exponential(size=E) * (rng.random(E) < 0.8) + 1e-9
    return table(rows, rng.multinomial(rows - tail, p / p.sum()), tail)


def operands(rows, E, H, n, dtype, how, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + rows + 31 * H + n)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x = layout(rnd(rows, H).to(dtype), how)
    w = layout((rnd(E, n, H) / H ** 0.5).to(dtype), how)
    return x, w, rnd


def poison(t, off, rows):
    """NaN where no expert reads."""
    if off is not None and off[-1] < rows:
        t[int(off[-1]):] = float("nan")
    return t


def dev(off):
    return None if off is None else torch.from_numpy(off).cuda()


def run_glu(rows, off, H, I, dtype, how="dense", act="silu", save=True, seed=0):
    E = 1 if off is None else len(off) - 1
    x, w, _ = operands(rows, E, H, 2 * I, dtype, how, seed)
    poison(x, off, rows)
    ref, kept = products.glu(np.nan_to_num(f64(x)), f64(w), off, act)
    a, gu = Out(dtype, how, rows, I), Out(dtype, how, rows, 2 * I) if save else None
    R().moe_glu(x, w if off is not None else w[0], a.t, gu.t if save else None, dev(off), act=act_kind(act))
    a.check("a", ref["a"], kept)
    if save:
        gu.check("gu", ref["gu"], kept)


def run_glu_backward(rows, off, H, I, dtype, how="dense", act="silu", dw_dtype=None, seed=0):
    E = 1 if off is None else len(off) - 1
    x, w, rnd = operands(rows, E, H, 2 * I, dtype, how, seed)
    gu, da = layout(rnd(rows, 2 * I).to(dtype), how), layout(rnd(rows, I).to(dtype), how)
    ref, kept = products.glu_backward(f64(da), f64(gu), f64(x), f64(w), off, act, UOUT[dtype])
    for t in (x, gu, da):
        poison(t, off, rows)
    dx, dw = Out(dtype, how, rows, H), Out(dw_dtype or dtype, "dense", E, 2 * I, H)
    ws = torch.empty(R().moe_glu_workspace(rows, E, H, I, fmt_of(dtype)), dtype=torch.uint8, device="cuda")
    R().moe_glu_backward(da, gu, x, w, dx.t, dw.t, ws, dev(off), act=act_kind(act))
    dx.check("dx", ref["dx"], kept)
    dw.check("dw", ref["dw"])


def run_linear(rows, off, K, N, dtype, how="dense", act="none", y_dtype=None, bias=True, residual=True, save=True, seed=0):
    E = 1 if off is None else len(off) - 1
    y_dtype = y_dtype or dtype
    x, w, rnd = operands(rows, E, K, N, dtype, how, seed)
    b = rnd(E, N) if bias else None
    r = layout(rnd(rows, N).to(y_dtype), how) if residual else None
    ref, kept = products.linear(f64(x), f64(w), f64(b), f64(r), off, act)
    poison(x, off, rows)
    y, z = Out(y_dtype, how, rows, N), Out(dtype, how, rows, N) if save else None
    R().moe_linear(x, w, y.t, b, r, z.t if save else None, dev(off), act=act_kind(act))
    y.check("y", ref["y"], kept)
    if save:
        z.check("z", ref["z"], kept)


def run_linear_backward(rows, off, K, N, dtype, how="dense", act="none", y_dtype=None, dw_dtype=None, seed=0):
    E = 1 if off is None else len(off) - 1
    y_dtype = y_dtype or dtype
    x, w, rnd = operands(rows, E, K, N, dtype, how, seed)
    dy, z = layout(rnd(rows, N).to(y_dtype), how), layout(rnd(rows, N).to(dtype), how)
    u_op = UOUT[dtype] if act != "none" or y_dtype != dtype else 0.0
    ref, kept = products.linear_backward(f64(dy), f64(z), f64(x), f64(w), off, act, u_op)
    for t in (x, z, dy):
        poison(t, off, rows)
    dx, dw, db = Out(dtype, how, rows, K), Out(dw_dtype or dtype, "dense", E, N, K), Out(F, "dense", E, N)
    ws = torch.empty(R().moe_linear_workspace(rows, E, K, N, fmt_of(dtype)), dtype=torch.uint8, device="cuda")
    R().moe_linear_backward(dy, z if act != "none" else None, x, w, dx.t, dw.t, db.t, ws, dev(off), act=act_kind(act))
    dx.check("dx", ref["dx"], kept)
    dw.check("dw", ref["dw"])
    db.check("dbias", ref["dbias"])


ALL = [run_glu, run_glu_backward, run_linear, run_linear_backward]
each = pytest.mark.parametrize("run", ALL, ids=lambda f: f.__name__)
types = pytest.mark.parametrize("dtype", [B, F], ids=["bf16", "f32"])
hows = pytest.mark.parametrize("how", ["dense", "gaps", "odd"])

DENSE = [(1, 64, 64), (1, 2048, 512), (2, 1, 1), (3, 7, 5), (17, 100, 36), (33, 64, 192), (64, 256, 128), (127, 63, 65),
         (128, 128, 128), (129, 72, 200), (300, 513, 130), (1000, 96, 257), (40, 2056, 72), (260, 328, 264)]


@each
@types
@pytest.mark.parametrize("rows,H,I", DENSE)
def test_one_weight(run, dtype, rows, H, I):
    run(rows, None, H, I, dtype)


@each
@types
@hows
@pytest.mark.parametrize("rows,H,I", [(70, 136, 72), (131, 65, 99)])
def test_layouts(run, dtype, how, rows, H, I):
    run(rows, None, H, I, dtype, how)
    run(rows, uneven(rows, 5, tail=9), H, I, dtype, how)


@each
@types
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_activations(run, dtype, act):
    run(90, uneven(90, 4), 128, 96, dtype, act=act)


GROUPS = [(1, 1, 0), (1, 256, 0), (5, 3, 0), (32, 256, 0), (64, 2, 1), (200, 7, 13), (500, 16, 0), (600, 600, 5), (1024, 1024, 0),
          (777, 1, 100), (900, 130, 30)]


@each
@types
@pytest.mark.parametrize("rows,E,tail", GROUPS)
def test_experts(run, dtype, rows, E, tail):
    run(rows, uneven(rows, E, tail), 72, 40, dtype)


@each
@types
@pytest.mark.parametrize("which", ["one", "last", "none", "first row", "edges"])
def test_skewed_experts(run, dtype, which):
    rows, E = 400, 9
    sizes = {"one": [0] * 4 + [400] + [0] * 4, "last": [0] * 8 + [400], "none": [0] * 9, "first row": [1] + [0] * 8,
             "edges": [127, 1, 128, 0, 0, 129, 0, 15, 0]}[which]
    run(rows, table(rows, sizes, rows - sum(sizes)), 64, 72, dtype)


@types
def test_formats_of_outputs(dtype):
    off = uneven(150, 6, 4)
    run_linear(150, off, 96, 80, dtype, y_dtype=F)
    run_linear(150, off, 96, 80, dtype, y_dtype=B, act="silu")
    run_linear(150, None, 96, 80, dtype, bias=False, residual=False, save=False)
    run_linear(150, None, 96, 80, dtype, bias=False, y_dtype=F)
    run_linear_backward(150, off, 96, 80, dtype, y_dtype=F)
    run_linear_backward(150, off, 96, 80, dtype, y_dtype=B, act="gelu")
    run_linear_backward(150, off, 96, 80, dtype, dw_dtype=F)
    run_linear_backward(150, off, 96, 80, dtype, dw_dtype=B)
    run_glu_backward(150, off, 96, 80, dtype, dw_dtype=F)
    run_glu_backward(150, off, 96, 80, dtype, dw_dtype=B)
    run_glu(150, off, 96, 80, dtype, save=False)


@each
def test_model_sizes(run):
    """The A3B shape over sixteen experts, and a piece of the DSV4 shape."""
    run(1100, uneven(1100, 16, 50), 2048, 512, B)
    run(300, None, 1024, 2048, B)


# larger sizes: many rows, few rows of long sums (split over the k), many small experts.  (The sizes that take each
# kernel and tile are product_sizes.py's.)
BIG = [(2048, 0, 1024, 1024), (1300, 0, 2048, 2048), (700, 0, 520, 1032), (20, 0, 4096, 512), (600, 40, 512, 256), (3000, 6, 512, 768)]


@each
@types
@pytest.mark.parametrize("rows,E,H,I", BIG)
def test_larger_products(run, dtype, rows, E, H, I):
    run(rows, uneven(rows, E, 7) if E else None, H, I, dtype)


# few rows: each over a long sum, with and without experts, sizes at the edges of its workgroups
FEW = [(1, 0, 2048, 512), (1, 0, 4096, 100), (3, 0, 1024, 17), (16, 0, 2056, 64), (17, 0, 2048, 40), (50, 0, 4096, 24), (6, 4, 2048, 72),
       (20, 9, 1024, 48), (40, 2, 4096, 33)]


@pytest.mark.parametrize("run", [run_glu, run_linear])
@types
@hows
@pytest.mark.parametrize("rows,E,H,I", FEW)
def test_few_rows(run, dtype, how, rows, E, H, I):
    run(rows, uneven(rows, E, rows // 6) if E else None, H, I, dtype, how, act="gelu")


# gradients of few tiles with a long k: few rows of many outputs (dx), many rows of small weights (dw)
LONG = [(1, 0, 0, 24, 4000), (3, 0, 0, 117, 2001), (40, 4, 3, 64, 1999), (65, 0, 0, 130, 1536), (2100, 0, 0, 72, 64), (2100, 0, 0, 65, 99),
        (3000, 3, 200, 40, 33), (5000, 2, 0, 9, 200)]


@pytest.mark.parametrize("run", [run_glu_backward, run_linear_backward])
@types
@hows
@pytest.mark.parametrize("rows,E,tail,H,I", LONG)
def test_long_sums(run, dtype, how, rows, E, tail, H, I):
    run(rows, uneven(rows, E, tail) if E else None, H, I, dtype, how, act="silu")


@types
def test_long_bias_sums(dtype):
    """A bias over so many rows that its gradient is summed in splits."""
    run_linear_backward(3000, None, 8, 70, dtype, act="silu")
    run_linear_backward(5000, uneven(5000, 2, 77), 16, 24, dtype)


def test_outputs_left_out():
    """Each gradient alone is the one that comes with the others; what it does not need may be missing."""
    L = R()
    rows, E, H, I = 130, 3, 72, 56
    off = dev(uneven(rows, E, 5))
    x, w, rnd = operands(rows, E, H, 2 * I, B, "dense")
    gu, da = rnd(rows, 2 * I).to(B), rnd(rows, I).to(B)
    ws = torch.empty(L.moe_glu_workspace(rows, E, H, I, L.MOE_AFMT_BF16), dtype=torch.uint8, device="cuda")
    new = lambda *s, dt=B: torch.full(s, FILL, dtype=dt, device="cuda")  # noqa: E731
    dx, dw = new(rows, H), new(E, 2 * I, H)
    L.moe_glu_backward(da, gu, x, w, dx, dw, ws, off)
    dx1, dw1 = new(rows, H), new(E, 2 * I, H)
    L.moe_glu_backward(da, gu, None, w, dx1, None, ws, off)
    L.moe_glu_backward(da, gu, x, None, None, dw1, ws, off)
    assert torch.equal(dx, dx1) and torch.equal(dw, dw1)
    w2, dy, z = w[:, :I].contiguous(), rnd(rows, I).to(B), rnd(rows, I).to(B)
    ws = torch.empty(L.moe_linear_workspace(rows, E, H, I, L.MOE_AFMT_BF16), dtype=torch.uint8, device="cuda")
    for act in (L.MOE_ACT_NONE, L.MOE_ACT_GELU):
        outs = [[new(rows, H), new(E, I, H), new(E, I, dt=F)] for _ in range(2)]
        L.moe_linear_backward(dy, z, x, w2, *outs[0], ws, off, act=act)
        L.moe_linear_backward(dy, z, None, w2, outs[1][0], None, None, ws, off, act=act)
        L.moe_linear_backward(dy, z, x, None, None, outs[1][1], None, ws, off, act=act)
        L.moe_linear_backward(dy, z, None, None, None, None, outs[1][2], ws, off, act=act)
        assert all(torch.equal(p, q) for p, q in zip(*outs))


def test_residual_in_place():
    L = R()
    x, w, rnd = operands(77, 1, 64, 48, B, "dense")
    h = layout(rnd(77, 48), "gaps")
    want = torch.empty(77, 48, device="cuda")
    L.moe_linear(x, w[0], want, residual=h)
    L.moe_linear(x, w[0], h, residual=h)
    assert torch.equal(h, want)


def test_weights_are_views_of_records():
    """gate | up and down of the library's bf16 expert records, used where they lie."""
    L = R()
    E, H, I, rows = 4, 64, 128, 90
    record = torch.randn(E, 3 * H * I, device="cuda").to(B)
    wgu, wd = record[:, :2 * H * I].view(E, 2 * I, H), record[:, 2 * H * I:].view(E, H, I)
    assert wgu.data_ptr() == record.data_ptr() and not wgu.is_contiguous()
    off, x = dev(uneven(rows, E)), torch.randn(rows, H, device="cuda").to(B)
    outs = []
    for a, b in ((wgu, wd), (wgu.contiguous(), wd.contiguous())):
        act, y = torch.empty(rows, I, device="cuda", dtype=B), torch.empty(rows, H, device="cuda", dtype=B)
        L.moe_glu(x, a, act, offsets=off)
        L.moe_linear(act, b, y, offsets=off)
        outs.append((act, y))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_tables_that_are_no_offsets_write_nothing_outside():
    L = R()
    rows, E, H, I = 100, 6, 64, 64
    x, w, rnd = operands(rows, E, H, 2 * I, B, "dense")
    for bad in ([-(2 ** 31), 50, 20, 2 ** 31 - 1, 0, 100, 100], [100, 0, 100, 0, 100, 0, 100], [7] * 7, [2 ** 31 - 1] * 7,
                [0, 100, 200, 300, 400, 500, 600]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        buf = torch.full((rows + 20, I), FILL, dtype=B, device="cuda")
        L.moe_glu(x, w, buf[10:10 + rows], offsets=off)
        assert (buf[:10] == FILL).all() and (buf[10 + rows:] == FILL).all()
        ws = torch.empty(L.moe_glu_workspace(rows, E, H, I, L.MOE_AFMT_BF16), dtype=torch.uint8, device="cuda")
        dxb, dw = torch.full((rows + 20, H), FILL, dtype=B, device="cuda"), torch.empty(E, 2 * I, H, device="cuda", dtype=B)
        L.moe_glu_backward(rnd(rows, I).to(B), rnd(rows, 2 * I).to(B), x, w, dxb[10:10 + rows], dw, ws, off)
        assert (dxb[:10] == FILL).all() and (dxb[10 + rows:] == FILL).all() and torch.isfinite(dw).all()


def test_far_offsets():
    """Rows, experts and outputs past 2^31 elements from the first."""
    L = R()
    H, I, rows = 64, 64, 130
    ld = (1 << 31) // 100 // 8 * 8
    xs = torch.empty(rows * ld, dtype=B, device="cuda").view(rows, ld)[:, :H]
    xs.copy_(torch.randn(rows, H, device="cuda"))
    gs = (1 << 31) + 512
    ws = torch.empty(gs + 2 * I * H, dtype=B, device="cuda")
    w = torch.as_strided(ws, (2, 2 * I, H), (gs, H, 1))
    w.copy_(torch.randn(2, 2 * I, H, device="cuda") / 8)
    off = dev(table(rows, [60, 70]))
    a = torch.empty(rows * ld, dtype=B, device="cuda").view(rows, ld)[:, :I]
    want = torch.empty(rows, I, dtype=B, device="cuda")
    L.moe_glu(xs, w, a, offsets=off)
    L.moe_glu(xs.contiguous(), w.contiguous(), want, offsets=off)
    assert torch.equal(a, want)
    gu, da = torch.randn(rows, 2 * I, device="cuda").to(B), torch.randn(rows, I, device="cuda").to(B)
    wk = torch.empty(L.moe_glu_workspace(rows, 2, H, I, L.MOE_AFMT_BF16), dtype=torch.uint8, device="cuda")
    outs = []
    for x1, w1, dx in ((xs, w, a), (xs.contiguous(), w.contiguous(), torch.empty(rows, H, dtype=B, device="cuda"))):
        dw = torch.empty(2, 2 * I, H, dtype=B, device="cuda")
        L.moe_glu_backward(da, gu, x1, w1, dx, dw, wk, off)
        outs.append((dx.clone(), dw))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_not_finite_stays_in_its_row():
    """NaN and infinities of one row of x reach that row's outputs alone; of dropped rows, none."""
    L = R()
    rows, H, I = 70, 40, 24
    for dtype in (B, F):
        x, w, rnd = operands(rows, 1, H, 2 * I, dtype, "dense")
        a, b = (torch.empty(rows, I, dtype=dtype, device="cuda") for _ in range(2))
        L.moe_glu(x, w, a)
        x2 = x.clone()
        x2[13, 5] = float("nan")
        x2[40, 0] = float("inf")
        L.moe_glu(x2, w, b)
        good = torch.ones(rows, dtype=torch.bool)
        good[[13, 40]] = False
        assert torch.equal(a[good], b[good]) and b[13].isnan().all() and not b[40].isfinite().any()


def step(L, s):
    """A training step of a block of experts between dispatch and combine, forward and back."""
    T, k, E = s["T"], s["k"], s["E"]
    L.moe_dispatch(s["idx"], E, s["x"], s["xs"], s["perm"], s["inv"], s["off"], s["wsd"])
    L.moe_glu(s["xs"], s["w1"], s["a"], s["gu"], s["off"])
    L.moe_linear(s["a"], s["w2"], s["ys"], s["b2"], offsets=s["off"])
    L.moe_combine(s["ys"], s["inv"], s["gate"], s["y"])
    # a shared expert on every token, added in place
    L.moe_glu(s["x"], s["v1"], s["sa"], s["sgu"])
    L.moe_linear(s["sa"], s["v2"], s["y"], residual=s["y"])
    L.moe_combine_backward(s["dy"], s["ys"], s["inv"], s["gate"], s["dys"], s["dgate"])
    L.moe_linear_backward(s["dys"], None, s["a"], s["w2"], s["da"], s["dw2"], s["db2"], s["wsl"], s["off"])
    L.moe_glu_backward(s["da"], s["gu"], s["xs"], s["w1"], s["dxs"], s["dw1"], s["wsg"], s["off"])
    L.moe_dispatch_backward(s["dxs"], s["inv"], s["dx"])


def step_state(L, T=96, k=2, E=5, H=72, I=40, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    P = T * k
    new = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.int32)  # noqa: E731
    u8 = lambda n: torch.empty(max(n, 1), device="cuda", dtype=torch.uint8)  # noqa: E731
    idx = torch.randint(-1, E, (T, k), device="cuda", generator=g, dtype=torch.int32)
    s = dict(T=T, k=k, E=E, H=H, I=I, idx=idx, x=rnd(T, H), w1=rnd(E, 2 * I, H) / H ** 0.5, w2=rnd(E, H, I) / I ** 0.5, b2=rnd(E, H),
             v1=rnd(2 * I, H) / H ** 0.5, v2=rnd(H, I) / I ** 0.5, gate=torch.rand(T, k, device="cuda", generator=g), dy=rnd(T, H),
             xs=new(P, H), perm=i32(P), inv=i32(T, k), off=i32(E + 1), wsd=u8(L.moe_dispatch_workspace(T, k, E)),
             a=new(P, I), gu=new(P, 2 * I), ys=new(P, H), y=new(T, H), sa=new(T, I), sgu=new(T, 2 * I), dys=new(P, H),
             dgate=new(T, k), da=new(P, I), dw2=new(E, H, I), db2=new(E, H), wsl=u8(L.moe_linear_workspace(P, E, I, H, L.MOE_AFMT_F32)),
             dxs=new(P, H), dw1=new(E, 2 * I, H), wsg=u8(L.moe_glu_workspace(P, E, H, I, L.MOE_AFMT_F32)), dx=new(T, H))
    return s


OUTS = ("y", "dgate", "dw2", "db2", "dw1", "dx")


def test_a_training_step_against_autograd():
    """dispatch, glu, linear, combine, a shared expert, and all of it back, against fp64 autograd of the dense form.
    The steps are fp32: 2e-5 of an output's largest value covers sums of a few hundred terms at 2^-24 each."""
    L = R()
    s = step_state(L)
    step(L, s)
    d = {n: s[n].double().cpu().requires_grad_() for n in ("x", "w1", "w2", "b2", "gate", "v1", "v2")}
    silu = torch.nn.functional.silu
    I = s["I"]

    def block(x, w1, w2, b):
        gu = x @ w1.T
        return (silu(gu[:, :I]) * gu[:, I:]) @ w2.T + b

    y = 0
    idx = s["idx"].cpu().long()
    for e in range(s["E"]):
        w = (d["gate"] * (idx == e)).sum(1, keepdim=True)
        y = y + w * block(d["x"], d["w1"][e], d["w2"][e], d["b2"][e])
    (y * s["dy"].double().cpu()).sum().backward()
    ref = {"y": (y + block(d["x"], d["v1"], d["v2"], 0.0)).detach(), "dw1": d["w1"].grad, "dw2": d["w2"].grad, "db2": d["b2"].grad,
           "dx": d["x"].grad, "dgate": d["gate"].grad}
    for n in OUTS:
        err = (s[n].double().cpu() - ref[n]).abs().max() / ref[n].abs().max()
        assert err < 2e-5, (n, float(err))


def test_replayed_graph_and_two_streams():
    L = R()
    states = [step_state(L, seed=i) for i in (1, 2)]
    want = []
    for s in states:
        step(L, s)
        want.append({n: s[n].clone() for n in OUTS})
    graphs = []
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(L, s)
        graphs.append(g)
    for turn in range(4):
        for s in states:
            for n in OUTS:
                s[n].fill_(FILL)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for s, w in zip(states, want):
            assert all(torch.equal(s[n], w[n]) for n in OUTS), turn
        step(L, states[turn % 2])
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, s in zip(streams, states):
            with torch.cuda.stream(st):
                step(L, s)
    torch.cuda.synchronize()
    for s, w in zip(states, want):
        assert all(torch.equal(s[n], w[n]) for n in OUTS)


# rows, experts, H, I: few rows; a long k in parts, of dx and of dw; both gradients in one launch; sizes of their own
CAPTURED = [(1, 0, 2048, 512), (3, 0, 64, 2000), (2100, 0, 65, 99), (130, 3, 72, 56), (1300, 5, 640, 512), (77, 2, 33, 1001)]


@types
@pytest.mark.parametrize("rows,E,H,I", CAPTURED)
def test_replayed_calls_need_nothing_of_their_workspaces(dtype, rows, E, H, I):
    """Every entry point in one graph: replays equal the eager run, whatever outputs and workspaces held before,
    with workspaces that start anywhere."""
    L = R()
    off = dev(uneven(rows, E, rows // 20)) if E else None
    n = max(E, 1)
    x, w, rnd = operands(rows, n, H, 2 * I, dtype, "dense")
    w, v = (w, rnd(n, H, I).to(dtype)) if E else (w[0], rnd(H, I).to(dtype))
    da, gu, dy, z = (rnd(rows, c).to(dtype) for c in (I, 2 * I, H, H))
    bias = rnd(n, H) if E else rnd(H)
    new = lambda *s, dt=dtype: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    outs = dict(a=new(rows, I), gu=new(rows, 2 * I), y=new(rows, H), z=new(rows, H), dx=new(rows, H), dw=torch.zeros_like(w),
                da=new(rows, I), dv=torch.zeros_like(v), db=torch.zeros_like(bias))
    wsg = torch.empty(L.moe_glu_workspace(rows, n, H, I, fmt_of(dtype)) + 5, dtype=torch.uint8, device="cuda")[5:]
    wsl = torch.empty(L.moe_linear_workspace(rows, n, I, H, fmt_of(dtype)) + 3, dtype=torch.uint8, device="cuda")[3:]

    def calls():
        L.moe_glu(x, w, outs["a"], outs["gu"], off)
        L.moe_linear(da, v, outs["y"], bias, None, outs["z"], off, act=L.MOE_ACT_GELU)
        L.moe_glu_backward(da, gu, x, w, outs["dx"], outs["dw"], wsg, off)
        L.moe_linear_backward(dy, z, da, v, outs["da"], outs["dv"], outs["db"], wsl, off, act=L.MOE_ACT_GELU)

    def refill():
        for t in outs.values():
            t.fill_(FILL)
        for t in (wsg, wsl):
            t.fill_(255)

    refill()
    calls()
    want = {k: t.clone() for k, t in outs.items()}
    assert all(torch.isfinite(t).all() for t in want.values())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for turn in range(4):
        refill()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(outs[k], want[k]) for k in outs), turn
        refill()
        calls()
        assert all(torch.equal(outs[k], want[k]) for k in outs), turn
