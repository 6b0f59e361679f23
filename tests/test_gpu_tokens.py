"""GPU: tokens sorted by expert, moved, weighted and brought back, their gradients and the gates' gradient,
against the fp64 definitions; bounds are derived per element.

An fp32 operation errs by at most U32 = 2^-24 of its result, a rounding to bf16 by 2^-8; a sum whose
terms pass through at most n additions errs by n * U32 times the sum of magnitudes."""
import numpy as np
import pytest
import torch

from oracle import tokens

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
UOUT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F, B = torch.float32, torch.bfloat16


def R():
    import routed_expert_ffn_02_amd
    return routed_expert_ffn_02_amd


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


def within(got, ref, err, dtype):
    """|got - ref| <= err + the output's own rounding of a value up to |ref| + err."""
    got = f64(got)
    tol = err + UOUT[dtype] * (np.abs(ref) + err) + 1e-37
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), float((np.abs(got - ref) / tol).max()), np.argwhere(bad)[:4].tolist())


def routing(T, k, E, drop, seed=0):
    rng = np.random.default_rng(seed + 131 * T + k)
    idx = rng.integers(0, E, size=(T, k)).astype(np.int32)
    out = rng.random((T, k)) < drop
    idx[out] = rng.choice(np.array([-1, E, -(2 ** 31), 2 ** 31 - 1], np.int32), size=int(out.sum()))
    if drop and T > 2:
        idx[T // 2] = -1                      # a token without any expert
    return idx


def run_dispatch(idx, E, x, tail=-7):
    """All outputs of moe_dispatch on prefilled buffers."""
    T, k = idx.shape
    H = x.shape[1]
    xs = torch.full((T * k, H), 77.0, dtype=x.dtype, device="cuda")
    perm = torch.full((T * k,), tail, dtype=torch.int32, device="cuda")
    inv = torch.full((T, k), tail, dtype=torch.int32, device="cuda")
    off = torch.full((E + 1,), tail, dtype=torch.int32, device="cuda")
    ws = torch.empty(R().moe_dispatch_workspace(T, k, E), dtype=torch.uint8, device="cuda")
    R().moe_dispatch(dev(idx), E, x, xs, perm, inv, off, ws)
    return xs, perm, inv, off


def check_dispatch(idx, E, x, got):
    T, k = idx.shape
    xs, perm, inv, off = got
    flat = idx.reshape(-1)
    kept = (flat >= 0) & (flat < E)
    # the definition, by a stable sort of the kept pairs (tokens.sort_pairs is its slow form)
    order = np.flatnonzero(kept)[np.argsort(flat[kept], kind="stable")]
    n = len(order)
    rinv = np.full(T * k, -1)
    rinv[order] = np.arange(n)
    assert np.array_equal(perm[:n].cpu().numpy(), order)
    assert (perm[n:] == -7).all()
    assert np.array_equal(inv.cpu().numpy().reshape(-1), rinv)
    assert np.array_equal(off.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(flat[kept], minlength=E))]))
    assert torch.equal(xs[:n], x[dev(order // k)])
    assert (xs[n:] == 77.0).all()             # rows behind the last pair


SORTS = [(1, 1, 1, 0.0), (1, 2, 8, 0.0), (1, 8, 256, 0.0), (3, 5, 7, 0.3), (4, 8, 256, 0.0), (64, 8, 256, 0.1),
         (127, 1, 2, 0.0), (130, 6, 1000, 0.02), (97, 16, 1024, 0.0), (300, 7, 33, 0.5), (1024, 8, 256, 0.0),
         (2049, 3, 255, 0.01), (4096, 8, 256, 0.02), (9001, 16, 512, 0.0), (5000, 30, 64, 0.1), (700, 100, 1000, 0.1),
         (11, 1024, 1024, 0.2), (1024, 1, 16, 0.0), (341, 3, 8, 0.1), (2048, 4, 100, 0.0), (8193, 1, 5, 0.0), (70001, 8, 3, 0.1),
         (300007, 2, 1024, 0.02), (20000, 4, 1, 0.3)]


@pytest.mark.parametrize("T,k,E,drop", SORTS)
def test_sort(T, k, E, drop):
    idx = routing(T, k, E, drop)
    x = torch.arange(T * 4, device="cuda", dtype=torch.float32).reshape(T, 4)
    got = run_dispatch(idx, E, x)
    check_dispatch(idx, E, x, got)
    if T * k <= 600:
        perm, inv, off = tokens.sort_pairs(idx, E)
        assert np.array_equal(got[2].cpu().numpy(), inv) and np.array_equal(got[3].cpu().numpy(), off)


@pytest.mark.parametrize("E", [1, 2, 64, 1024])
@pytest.mark.parametrize("which", ["one expert", "none kept", "last only", "runs"])
def test_sort_skewed(E, which):
    T, k = 1500, 3
    idx = {"one expert": np.full((T, k), E - 1), "none kept": np.full((T, k), -1),
           "last only": np.where(np.arange(T * k).reshape(T, k) == T * k - 1, 0, E),
           "runs": (np.arange(T * k).reshape(T, k) // 97) % E}[which].astype(np.int32)
    x = torch.randn(T, 8, device="cuda")
    check_dispatch(idx, E, x, run_dispatch(idx, E, x))


def test_sort_alone():
    T, k, E = 500, 4, 32
    idx = routing(T, k, E, 0.1)
    perm, inv, off = (torch.full(s, -7, dtype=torch.int32, device="cuda") for s in ((T * k,), (T, k), (E + 1,)))
    ws = torch.empty(R().moe_dispatch_workspace(T, k, E), dtype=torch.uint8, device="cuda")
    R().moe_dispatch(dev(idx), E, None, None, perm, inv, off, ws)
    x = torch.zeros(T, 1, device="cuda")
    want = run_dispatch(idx, E, x)
    assert torch.equal(perm, want[1]) and torch.equal(inv, want[2]) and torch.equal(off, want[3])


SHAPES = [(1, 1, 1), (1, 8, 2048), (2, 3, 7), (4, 6, 4096), (5, 2, 63), (7, 9, 513), (33, 8, 1000), (64, 17, 65), (50, 4, 2056),
          (129, 2, 1999), (19, 1, 8200)]


def views(t, how):
    """The values of t in a layout: dense, rows with gaps, or starting one element off 16 bytes."""
    if how == "dense":
        return t
    T, H = t.shape
    pad, first = (24, 8) if how == "gaps" else (3, 1)
    buf = torch.full((T, H + pad), 55.0, dtype=t.dtype, device="cuda")
    buf[:, first:first + H] = t
    return buf[:, first:first + H]


def around(view):
    """The bytes of the buffer behind a view that are not the view's own."""
    base = view._base
    if base is None:
        return torch.zeros(0, device="cuda")
    mask = torch.ones_like(base, dtype=torch.bool)
    off = view.storage_offset()
    mask[:, off:off + view.shape[1]] = False
    return base[mask]


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("T,k,H", SHAPES)
def test_move(T, k, H, dtype):
    E = 16
    idx = routing(T, k, E, 0.1 if T > 4 else 0.0)
    x = torch.randn(T, H, device="cuda").to(dtype)
    for how in ("dense", "gaps", "odd"):
        check_dispatch(idx, E, x, run_dispatch(idx, E, views(x, how)))


@pytest.mark.parametrize("out", [F, B])
@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("T,k,H", SHAPES)
def test_combine_and_dispatch_backward(T, k, H, dtype, out):
    inv = tokens.sort_pairs(routing(T, k, 16, 0.2 if T > 4 else 0.0), 16)[1]
    rng = np.random.default_rng(H)
    ys = torch.randn(T * k, H, device="cuda").to(dtype)
    w = rng.random((T, k)).astype(np.float32)
    w[inv < 0] = np.nan                        # a pair left out: its gate and every row without a pair unread
    ys[int(inv.max()) + 1:] = float("nan")
    for how in ("dense", "gaps", "odd"):
        y = views(torch.full((T, H), 9.0, dtype=out, device="cuda"), how)
        R().moe_combine(ys, dev(inv), dev(w), y)
        ref, mag = tokens.gather_sum(f64(ys), inv, w)
        within(y, ref, (k + 1) * U32 * mag, out)
        assert (around(y) == 55.0).all()
        dx = views(torch.full((T, H), 9.0, dtype=out, device="cuda"), how)
        R().moe_dispatch_backward(ys, dev(inv), dx)
        ref, mag = tokens.gather_sum(f64(ys), inv)
        within(dx, ref, k * U32 * mag, out)
        assert (around(dx) == 55.0).all()


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("grad", [F, B])
@pytest.mark.parametrize("T,k,H", SHAPES)
def test_combine_backward(T, k, H, grad, dtype):
    inv = tokens.sort_pairs(routing(T, k, 16, 0.2 if T > 4 else 0.0), 16)[1]
    w = np.random.default_rng(H).random((T, k)).astype(np.float32)
    w[inv < 0] = np.nan
    ys = torch.randn(T * k, H, device="cuda").to(dtype)
    ys[int(inv.max()) + 1:] = float("nan")
    g = torch.randn(T, H, device="cuda").to(grad)
    rdys, written, rdw, mag = tokens.combine_backward(f64(g), f64(ys), inv, w)
    wr = torch.from_numpy(written).cuda()
    # a row's dot product: at most H additions in any order (64 and more of them side by side)
    depth = 8 * -(-H // 512) + 16
    for how in ("dense", "gaps", "odd"):
        dy = views(g, how)
        dys = torch.full_like(ys, 77.0)
        dw = torch.full((T, k), 9.0, device="cuda")
        R().moe_combine_backward(dy, ys, dev(inv), dev(w), dys, dw)
        within(dys[wr], rdys[written], U32 * np.abs(rdys[written]), dtype)
        assert (dys[~wr] == 77.0).all()
        within(dw, rdw, depth * U32 * mag, F)
    # either output alone, and dys in ys's place: the same bits
    one, two, both = torch.full_like(dys, 77.0), torch.empty_like(dw), ys.clone()
    R().moe_combine_backward(g, None, dev(inv), dev(w), one, None)
    R().moe_combine_backward(g, ys, dev(inv), None, None, two)
    assert torch.equal(one, dys) and torch.equal(two, dw)
    R().moe_combine_backward(g, both, dev(inv), dev(w), both, two)
    assert torch.equal(both[wr], dys[wr]) and torch.equal(two, dw)


def test_tables_out_of_range_are_left_out():
    """inv entries that name no row (a table the library did not write) count as pairs left out."""
    T, k, H = 6, 3, 40
    inv = np.array([[0, 18, 2], [-5, 1, 2 ** 31 - 1], [3, 4, 5], [-(2 ** 31), 6, 7], [8, 9, 100], [10, 11, -1]], np.int32)
    ys, w = torch.randn(T * k, H, device="cuda"), torch.rand(T, k, device="cuda")
    y = torch.empty(T, H, device="cuda")
    R().moe_combine(ys, dev(inv), w, y)
    ref, mag = tokens.gather_sum(f64(ys), inv, f64(w))
    within(y, ref, (k + 1) * U32 * mag, F)
    dys, dw = torch.full_like(ys, 77.0), torch.empty_like(w)
    R().moe_combine_backward(y, ys, dev(inv), w, dys, dw)
    rdys, written, rdw, mag = tokens.combine_backward(f64(y), f64(ys), inv, f64(w))
    wr = torch.from_numpy(written).cuda()
    within(dys[wr], rdys[written], U32 * np.abs(rdys[written]), F)
    assert (dys[~wr] == 77.0).all()
    within(dw, rdw, 32 * U32 * mag, F)


def test_infinities_and_nan_follow_the_formula():
    ys = torch.tensor([[1.0, float("inf"), float("nan"), -float("inf")], [2.0, 1.0, 1.0, float("inf")]], device="cuda")
    inv = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    for dtype in (F, B):
        y = torch.empty(1, 4, dtype=dtype, device="cuda")
        R().moe_combine(ys.to(dtype), inv, torch.ones(1, 2, device="cuda"), y)
        assert y[0, 0] == 3 and y[0, 1] == float("inf") and y[0, 2].isnan() and y[0, 3].isnan()


def test_offsets_past_32_bits():
    """2^31 elements and more in the sorted rows: the last rows land where they belong."""
    H, k = 4096, 8
    T = (1 << 31) // (H * k) + 40
    E = 16
    g = torch.Generator(device="cuda").manual_seed(0)
    idx = torch.randint(0, E, (T, k), device="cuda", dtype=torch.int32, generator=g)
    x = torch.randint(-100, 100, (T, H), device="cuda", dtype=torch.int16, generator=g).view(B)
    xs = torch.zeros(T * k, H, dtype=B, device="cuda")
    perm, inv, off = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((T * k,), (T, k), (E + 1,)))
    ws = torch.empty(R().moe_dispatch_workspace(T, k, E), dtype=torch.uint8, device="cuda")
    R().moe_dispatch(idx, E, x, xs, perm, inv, off, ws)
    order = torch.argsort(idx.reshape(-1).long(), stable=True)
    assert torch.equal(perm.long(), order)
    bits, src = xs.view(torch.int16), x.view(torch.int16)
    for lo in range(0, T * k, 1 << 17):
        assert torch.equal(bits[lo:lo + (1 << 17)], src[order[lo:lo + (1 << 17)] // k])
    # back: k equal rows each, an exact sum in fp32 of small whole numbers
    xs.copy_(torch.ones((), dtype=B, device="cuda"))
    xs[-1] = 3.0
    dx = torch.empty(T, H, device="cuda")
    R().moe_dispatch_backward(xs, inv, dx)
    want = torch.full((T,), float(k), device="cuda")
    want[order[-1] // k] += 2
    assert torch.equal(dx, want[:, None].expand(T, H))
    w = torch.full((T, k), 0.5, device="cuda")
    dw = torch.empty(T, k, device="cuda")
    R().moe_combine_backward(dx, xs, inv, w, xs, dw)
    assert torch.equal(xs[-1].float(), (want[order[-1] // k] * 0.5).expand(H))
    assert dw.reshape(-1)[order[-1]].item() == 3.0 * H * (k + 2)
    assert dw.reshape(-1)[order[0]].item() == H * want[order[0] // k].item()


# --- the gates' gradient -----------------------------------------------------
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (5, 2, 8), (6, 3, 65), (37, 8, 100), (64, 6, 256), (9, 16, 257),
                                   (21, 16, 1000), (8, 64, 1024), (3, 1000, 1024),
                                   (5, 150, 40), (70, 12, 5)])
def test_topk_backward(T, k, E, renorm):
    rng = np.random.default_rng(E + k + renorm)
    z = (3.0 * rng.standard_normal((T, E))).astype(np.float32)
    idx = np.stack([rng.permutation(E)[:k] if k <= E else rng.integers(0, E, k) for _ in range(T)]).astype(np.int32)
    if T > 4:
        idx[1, 0] = idx[1, k - 1]                 # the same expert twice (k >= 2 here)
        idx[2, 0] = -1
        idx[3] = E                                # no pair kept
        z[4] = -np.inf                            # every logit masked
        z[0, idx[0, 0]] = -np.inf
        z[2, ::2] = -np.inf
    if T > 6:
        z[5, 1::2] = np.finfo(np.float32).min     # masks of the lowest finite value: no share either
        z[6] = np.finfo(np.float32).min           # all alike: every logit the same share
    dw = rng.standard_normal((T, k)).astype(np.float32)
    dw[(idx < 0) | (idx >= E)] = np.nan           # not read into anything
    got = torch.full((T, E), 9.0, device="cuda")
    zt = dev(z)
    R().moe_topk_backward(zt, dev(idx), dev(dw), renorm, got)
    ref, p, mag = tokens.topk_backward(z, idx, np.where(np.isnan(dw), 0, dw), renorm)
    # p_e = exp(z_e - m) / sum: the exponential errs by U32 |z_e - m| of the product with log2 e, and a few
    # roundings of its own; the sum's terms err alike and pass through at most E / 64 + 8 additions
    fin = np.where(np.isfinite(z), z, np.nan)
    span = np.nan_to_num(np.nanmax(np.where(np.isnan(fin), -1e30, fin), 1) - np.nanmin(np.where(np.isnan(fin), 1e30, fin), 1))
    span = np.clip(span, 0, 100)[:, None]
    rel = 2 * (2 * span + 8 + E / 64 + 8) * U32
    M = np.sum(p * mag, axis=1, keepdims=True)
    within(got, ref, p * (mag + M) * (2 * rel + (k + 24) * U32), F)
    R().moe_topk_backward(zt, dev(idx), dev(dw), renorm, zt)      # in place: the same bits
    assert torch.equal(zt, got)


def test_topk_backward_follows_the_gates():
    """moe_topk's own gates and choice, differentiated: differences of the library's forward pass in
    fp32 along a direction agree to the size that their rounding leaves."""
    import workloads as W
    from moe_harness import Harness
    r = R()
    T, E, k = 16, 64, 4
    for renorm in (0, 1):
        h = Harness(W.TINY.with_(n_experts=E, top_k=k, renorm=renorm), r.MOE_MODE_OFFLOAD, n_slots=1, max_tokens=T)
        z = torch.randn(T, E, device="cuda") * 2
        idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
        w = torch.empty(T, k, device="cuda")
        r.moe_topk(h.ctx, z, T, idx, w)
        dw, way = torch.randn(T, k, device="cuda"), torch.randn(T, E, device="cuda")
        dz = torch.empty(T, E, device="cuda")
        r.moe_topk_backward(z, idx, dw, renorm, dz)
        step, sides = 2.0 ** -7, []
        for s in (step, -step):
            i2, w2 = torch.empty_like(idx), torch.empty_like(w)
            r.moe_topk(h.ctx, z + s * way, T, i2, w2)
            # gates by expert, so that a swapped order of the same choice does not matter
            sides.append((torch.zeros(T, E, device="cuda").scatter_(1, i2.long(), w2), i2.sort(1).values))
        same = (sides[0][1] == idx.sort(1).values).all(1) & (sides[1][1] == idx.sort(1).values).all(1)
        assert same.sum() >= T // 4
        dense = torch.zeros(T, E, device="cuda").scatter_(1, idx.long(), dw)
        num = (dense * (sides[0][0] - sides[1][0])).sum(1) / (2 * step)
        ana = (dz * way).sum(1)
        # third-order term: step^2 / 6 times a third derivative of at most about 6 |dw| |way|^3 p; gates in fp32
        # err by 2^-22 or so, over 2 step
        size = dense.abs().sum(1)
        tol = size * (step ** 2 * way.abs().amax(1) ** 3 + 2.0 ** -20 / (2 * step))
        assert ((num - ana).abs() <= tol)[same].all()


# --- streams and graphs ------------------------------------------------------
@pytest.mark.parametrize("T", [100, 700, 3000])   # one for each form of the sort
def test_two_streams_at_once_and_graph_replays(T):
    """Calls that share nothing but inputs run at once on two streams; a captured sequence, replayed with
    eager work between, gives the eager bits each time on new inputs."""
    r = R()
    k, E, H = 8, 64, 512

    class Pass:
        def __init__(self, seed):
            self.g = torch.Generator(device="cuda").manual_seed(seed)
            self.idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
            self.x = torch.empty(T, H, dtype=B, device="cuda")
            self.w = torch.empty(T, k, device="cuda")
            self.xs = torch.zeros(T * k, H, dtype=B, device="cuda")
            self.perm, self.inv, self.off = (torch.zeros(s, dtype=torch.int32, device="cuda")
                                             for s in ((T * k,), (T, k), (E + 1,)))
            self.ws = torch.empty(r.moe_dispatch_workspace(T, k, E), dtype=torch.uint8, device="cuda")
            self.y, self.dw = torch.empty(T, H, device="cuda"), torch.empty(T, k, device="cuda")
            self.dys, self.dx = torch.zeros(T * k, H, dtype=B, device="cuda"), torch.empty(T, H, device="cuda")
            self.load()

        def load(self):
            self.idx.copy_(torch.randint(-1, E, (T, k), device="cuda", generator=self.g))
            self.x.copy_(torch.randn(T, H, device="cuda", generator=self.g))
            self.w.copy_(torch.rand(T, k, device="cuda", generator=self.g))

        def run(self, stream=None):
            r.moe_dispatch(self.idx, E, self.x, self.xs, self.perm, self.inv, self.off, self.ws, stream=stream)
            r.moe_combine(self.xs, self.inv, self.w, self.y, stream=stream)
            r.moe_combine_backward(self.y, self.xs, self.inv, self.w, self.dys, self.dw, stream=stream)
            r.moe_dispatch_backward(self.dys, self.inv, self.dx, stream=stream)

        def outputs(self):
            n = int(self.off[E])
            return [t.clone() for t in (self.xs[:n], self.perm[:n], self.inv, self.off, self.y, self.dw, self.dys[:n], self.dx)]

    a, b = Pass(1), Pass(2)
    a.run()
    b.run()
    torch.cuda.synchronize()
    want = a.outputs(), b.outputs()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        a.run(s1)
        b.run(s2)
    torch.cuda.synchronize()
    for got, ref in zip((a.outputs(), b.outputs()), want):
        assert all(torch.equal(p, q) for p, q in zip(got, ref))
    graphs = []
    for p in (a, b):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                p.run()
        graphs.append(g)
    for _ in range(3):
        for p, g, s in zip((a, b), graphs, (s1, s2)):
            p.load()
        torch.cuda.synchronize()
        for g, s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for p in (a, b):
            got = p.outputs()
            p.run()
            torch.cuda.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(got, p.outputs()))


def test_streams_and_devices_as_the_binding_takes_them():
    """A stream object, its handle and the current stream lead to the same call; a tensor on the host
    among tensors on the GPU is named."""
    r = R()
    inv = torch.tensor([[0, 1], [3, 2]], dtype=torch.int32, device="cuda")
    ys, w = torch.randn(4, 33, device="cuda"), torch.rand(2, 2, device="cuda")
    ys[2] = float("inf")
    out = [torch.empty(2, 33, device="cuda") for _ in range(4)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    r.moe_combine(ys, inv, w, out[0])
    r.moe_combine(ys, inv, w, out[1], stream=s)
    r.moe_combine(ys, inv, w, out[2], stream=s.cuda_stream)
    with torch.cuda.stream(s):
        r.moe_combine(ys, inv, w, out[3])
    torch.cuda.synchronize()
    assert all(torch.equal(o, out[0]) for o in out)
    for bad in (dict(ys=ys.cpu()), dict(inv=inv.cpu()), dict(w=w.cpu()), dict(y=out[0].cpu())):
        with pytest.raises(r.MoeError, match=f"{list(bad)[0]} must be on the GPU"):
            r.moe_combine(**{**dict(ys=ys, inv=inv, w=w, y=out[0]), **bad})
    for bad in ("0", 1 << 70):
        with pytest.raises(r.MoeError, match="stream"):
            r.moe_combine(ys, inv, w, out[0], stream=bad)
