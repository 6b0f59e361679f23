"""Pins of the fp64 definitions around the experts: the moves and the gates' gradient against
autograd in fp64 and differences, the norms' gradient likewise."""
import itertools

import numpy as np
import pytest
import torch

from oracle import norm, tokens


def _idx(rng, T, k, E, drop=0.2):
    idx = rng.integers(0, E, size=(T, k)).astype(np.int32)
    idx[rng.random((T, k)) < drop] = -1
    idx[0] = -1                      # a token without any expert
    return idx


def test_sort_pairs_by_hand():
    perm, inv, off = tokens.sort_pairs(np.array([[2, 0], [5, 2], [-1, 0]]), 4)   # 5 and -1 are left out
    assert perm.tolist() == [1, 5, 0, 3]
    assert inv.tolist() == [[2, 0], [-1, 3], [-1, 1]]
    assert off.tolist() == [0, 2, 2, 4, 4]


@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 3), (5, 3, 4, 7), (9, 2, 16, 5)])
def test_moves_are_autograd(T, k, E, H):
    rng = np.random.default_rng(T + k)
    idx = _idx(rng, T, k, E)
    if T == 1:
        idx[:] = 0
    perm, inv, _ = tokens.sort_pairs(idx, E)
    n = len(perm)
    x = torch.tensor(rng.standard_normal((T, H)), requires_grad=True)
    w = torch.tensor(rng.random((T, k)), requires_grad=True)
    a = torch.tensor(rng.standard_normal((n, H)))
    xs = x[torch.tensor(perm // k, dtype=torch.long)]
    assert np.array_equal(xs.detach().numpy(), tokens.dispatch(x.detach().numpy(), perm, k))
    ys = (xs * a).detach().requires_grad_()
    y = torch.zeros(T, H, dtype=torch.float64).index_add(
        0, torch.tensor(perm // k, dtype=torch.long), w.reshape(-1)[torch.tensor(perm, dtype=torch.long)][:, None] * ys)
    full = np.zeros((T * k, H))
    full[:n] = ys.detach().numpy()
    np.testing.assert_allclose(tokens.gather_sum(full, inv, w.detach().numpy())[0], y.detach().numpy(), atol=1e-13)
    dy = torch.tensor(rng.standard_normal((T, H)))
    gw, gys = torch.autograd.grad(y, (w, ys), dy)
    dys, written, dw, _ = tokens.combine_backward(dy.numpy(), full, inv, w.detach().numpy())
    assert written.sum() == n
    np.testing.assert_allclose(dys[:n], gys.numpy(), atol=1e-13)
    np.testing.assert_allclose(dw, gw.numpy(), atol=1e-13)
    dxs = rng.standard_normal((n, H))
    gx, = torch.autograd.grad(xs, x, torch.tensor(dxs))
    full[:n] = dxs
    np.testing.assert_allclose(tokens.gather_sum(full, inv)[0], gx.numpy(), atol=1e-13)


@pytest.mark.parametrize("renorm", [0, 1])
def test_gates_gradient_against_differences(renorm):
    rng = np.random.default_rng(3)
    T, k, E = 4, 3, 6
    z = rng.standard_normal((T, E))
    z[1, 2] = -np.inf
    z[2] = -np.inf
    idx = np.array([[0, 4, 2], [1, 2, 5], [0, 1, 2], [3, 3, -1]], np.int32)
    dw = rng.standard_normal((T, k))
    dz = tokens.topk_backward(z, idx, dw, renorm)[0]
    step = 1e-6
    for t, e in itertools.product(range(T), range(E)):
        if z[t, e] == -np.inf:
            assert dz[t, e] == 0
            continue
        hi, lo = z.copy(), z.copy()
        hi[t, e] += step
        lo[t, e] -= step
        num = np.sum(dw * (tokens.topk_gates(hi, idx, renorm) - tokens.topk_gates(lo, idx, renorm))) / (2 * step)
        assert abs(num - dz[t, e]) <= 1e-8, (t, e)      # differences: step^2 and 1e-16 / step


@pytest.mark.parametrize("post,gate,second", itertools.product((True, False), ("none", "token", "channel"), (True, False)))
def test_block_norm_gradient_against_differences_and_autograd(post, gate, second):
    rng = np.random.default_rng(11)
    T, H, alpha, eps = 3, 5, 0.7, 1e-3
    per_token = gate == "token"
    v = {"h": rng.standard_normal((T, H)), "y": rng.standard_normal((T, H))}
    v["y"][1] = 0.0                   # a row whose rms is eps alone
    if post:
        v["w_post"] = rng.standard_normal(H)
    if gate != "none":
        v["gate"] = rng.standard_normal(T if per_token else H)
    if second:
        v["w_pre"] = rng.standard_normal(H)
    dh, dx = rng.standard_normal((T, H)), rng.standard_normal((T, H))

    def loss(q):
        ho, xo = norm.block_norm(q["h"], q["y"], q.get("w_post"), q.get("gate"), per_token, q.get("w_pre"), alpha, eps)
        return np.sum(dh * ho) + (np.sum(dx * xo) if second else 0.0)

    h_out, _ = norm.block_norm(v["h"], v["y"], v.get("w_post"), v.get("gate"), per_token, None, alpha, eps)
    got = norm.block_norm_backward(h_out, v["y"], v.get("w_post"), v.get("gate"), per_token, v.get("w_pre"), dh,
                                   dx if second else None, alpha, eps)
    leaf = {n: torch.tensor(a, requires_grad=True) for n, a in v.items()}
    u = leaf["y"]
    if post:
        u = leaf["w_post"] * u / (u.pow(2).mean(1, keepdim=True) + eps).sqrt()
    g = leaf["gate"].reshape((T, 1) if per_token else (1, H)) if gate != "none" else 1.0
    ho = leaf["h"] + alpha * g * u
    total = (torch.tensor(dh) * ho).sum()
    if second:
        total = total + (torch.tensor(dx) * leaf["w_pre"] * ho / (ho.pow(2).mean(1, keepdim=True) + eps).sqrt()).sum()
    total.backward()
    for n, a in v.items():
        mine = got["d" + n][0]
        np.testing.assert_allclose(mine, leaf[n].grad.numpy(), rtol=1e-10, atol=1e-11)
        for i in np.ndindex(a.shape):
            if n == "y" and i[0] == 1 and post:
                continue              # curvature 1/eps: differences say nothing there
            step = 1e-6
            keep = a[i]
            a[i] = keep + step
            hi = loss(v)
            a[i] = keep - step
            lo = loss(v)
            a[i] = keep
            assert abs((hi - lo) / (2 * step) - mine[i]) <= 1e-6 * (1 + abs(mine[i])), (n, i)
