"""GPU: moves and sums of 128 MB of sorted rows and more, which pass by the caches: every format, the move
behind each form of the sort, widths that 8 does not divide, rows with gaps; against fp64 on the device."""
import pytest
import torch

from test_gpu_tokens import B, F, R, U32, UOUT, around, views

pytestmark = pytest.mark.gpu

# T, k, E, H: at least 128 MB of rows in bf16 (twice that in fp32); P <= 16384 and beyond; odd widths
CASES = [(2048, 8, 256, 4096), (12289, 4, 64, 1999), (4111, 8, 100, 2056), (5600, 6, 1000, 2051)]


def close(got, ref, mag, adds, dtype):
    """|got - ref| <= adds roundings of fp32 on the sum of magnitudes, and the output's own."""
    err = adds * U32 * mag
    bad = (got.double() - ref).abs() > err + UOUT[dtype] * (ref.abs() + err) + 1e-37
    assert not bad.any(), int(bad.sum())


def pairs(T, k, E, drop=0.1):
    g = torch.Generator(device="cuda").manual_seed(T + k)
    idx = torch.rand(T, E, device="cuda", generator=g).topk(k, 1).indices.int()
    idx[torch.rand(T, k, device="cuda", generator=g) < drop] = -1
    idx[T // 2] = E
    return idx.contiguous()


def sort(idx, E):
    """perm of the kept pairs and inv, by torch's stable sort."""
    key = torch.where((idx < 0) | (idx >= E), E, idx).reshape(-1).long()
    order = torch.argsort(key, stable=True)
    n = int((key < E).sum())
    inv = torch.full_like(order, -1)
    inv[order[:n]] = torch.arange(n, device="cuda")
    return order[:n], inv.int().reshape(idx.shape)


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("how", ["dense", "odd"])
@pytest.mark.parametrize("T,k,E,H", CASES)
def test_dispatch(T, k, E, H, dtype, how):
    idx = pairs(T, k, E)
    order, want = sort(idx, E)
    n = len(order)
    x = torch.randn(T, H, device="cuda").to(dtype)
    xs = torch.full((T * k, H), 77.0, dtype=dtype, device="cuda")
    assert xs.numel() * xs.element_size() >= 128 << 20
    perm, inv, off = (torch.full(s, -7, dtype=torch.int32, device="cuda") for s in ((T * k,), (T, k), (E + 1,)))
    ws = torch.empty(R().moe_dispatch_workspace(T, k, E), dtype=torch.uint8, device="cuda")
    R().moe_dispatch(idx, E, views(x, how), xs, perm, inv, off, ws)
    assert torch.equal(inv, want) and torch.equal(perm[:n].long(), order) and (perm[n:] == -7).all()
    assert torch.equal(xs[:n], x[order // k]) and (xs[n:] == 77.0).all() and off[E] == n


@pytest.mark.parametrize("out", [F, B])
@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("T,k,E,H", CASES)
def test_sums(T, k, E, H, dtype, out):
    idx = pairs(T, k, E)
    order, inv = sort(idx, E)
    rows = torch.randn(T * k, H, device="cuda").to(dtype)
    rows[len(order):] = float("nan")
    w = torch.rand(T, k, device="cuda")
    ref, mag = (torch.zeros(T, H, dtype=torch.float64, device="cuda") for _ in range(2))
    ref1, mag1 = torch.zeros_like(ref), torch.zeros_like(ref)
    for j in range(k):
        t = torch.nonzero(inv[:, j] >= 0)[:, 0]
        v = rows[inv[t, j].long()].double()
        ref1[t] += v
        mag1[t] += v.abs()
        v *= w[t, j, None].double()
        ref[t] += v
        mag[t] += v.abs()
    w[inv < 0] = float("nan")
    y, dx = (views(torch.full((T, H), 9.0, dtype=out, device="cuda"), how) for how in ("odd", "dense"))
    R().moe_combine(rows, inv, w, y)
    R().moe_dispatch_backward(rows, inv, dx)
    close(y, ref, mag, k + 1, out)
    close(dx, ref1, mag1, k, out)
    assert (around(y) == 55.0).all()


@pytest.mark.parametrize("grad", [F, B])
@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("T,k,E,H", CASES)
def test_combine_backward(T, k, E, H, dtype, grad):
    idx = pairs(T, k, E)
    order, inv = sort(idx, E)
    n = len(order)
    ys = torch.randn(T * k, H, device="cuda").to(dtype)
    w = torch.rand(T, k, device="cuda")
    dy = torch.randn(T, H, device="cuda").to(grad)
    dys, dw = torch.full_like(ys, 77.0), torch.full_like(w, 9.0)
    R().moe_combine_backward(dy, ys, inv, w, dys, dw)
    rdw, mag = (torch.zeros(T, k, dtype=torch.float64, device="cuda") for _ in range(2))
    for j in range(k):
        t = torch.nonzero(inv[:, j] >= 0)[:, 0]
        i = inv[t, j].long()
        v = w[t, j, None].double() * dy[t].double()
        close(dys[i], v, v.abs(), 1, dtype)
        v = ys[i].double() * dy[t].double()
        rdw[t, j], mag[t, j] = v.sum(1), v.abs().sum(1)
    assert (dys[n:] == 77.0).all()
    # a thread adds 8 products of each of its chunks of the row, 2048 elements apart, then lanes and wavefronts
    close(dw, rdw, mag, 8 * -(-H // 512) + 16, F)
    both, two = ys.clone(), torch.empty_like(dw)
    R().moe_combine_backward(dy, both, inv, w, both, two)        # in ys's place
    assert torch.equal(both[:n], dys[:n]) and torch.equal(two, dw)
