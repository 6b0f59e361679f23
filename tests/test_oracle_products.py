"""The oracle's products of the experts against differences and against torch in fp64."""
import numpy as np
import pytest
import torch

from oracle import products

OFF = [0, 3, 3, 7]   # three experts, the second without rows, the last row of eight without an expert


def case(seed=0, N=6):
    rng = np.random.default_rng(seed)
    return rng, rng.normal(size=(8, 5)), rng.normal(size=(3, N, 5)), rng


def torch_act(z, act):
    return {"none": lambda v: v, "silu": torch.nn.functional.silu,
            "gelu": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[act](z)


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_forward_against_torch(act):
    rng, x, w, _ = case()
    bias, res = rng.normal(size=(3, 6)), rng.normal(size=(8, 6))
    got, kept = products.linear(x, w, bias, res, OFF, act)
    glu, _ = products.glu(x, w, OFF, act)
    assert kept.tolist() == [True] * 7 + [False]
    for e, (lo, hi) in enumerate(products.ranges(OFF, 8)):
        z = torch.from_numpy(x[lo:hi] @ w[e].T)
        assert np.allclose(glu["a"][0][lo:hi], (torch_act(z[:, :3], act) * z[:, 3:]).numpy(), rtol=1e-12, atol=1e-14)
        z = z + torch.from_numpy(bias[e])
        assert np.allclose(got["y"][0][lo:hi], (torch_act(z, act) + torch.from_numpy(res[lo:hi])).numpy(), rtol=1e-12, atol=1e-14)
    assert (got["y"][0][7] == 0).all() and (glu["gu"][0][7] == 0).all()


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("which", ["glu", "linear"])
def test_gradients_against_differences(which, act):
    rng, x, w, _ = case(3)
    bias, g = rng.normal(size=(3, 6)), rng.normal(size=(8, 3 if which == "glu" else 6))

    def loss(x, w, bias):
        if which == "glu":
            return float((products.glu(x, w, OFF, act)[0]["a"][0] * g).sum())
        return float((products.linear(x, w, bias, None, OFF, act)[0]["y"][0] * g).sum())

    if which == "glu":
        got, _ = products.glu_backward(g, products.glu(x, w, OFF, act)[0]["gu"][0], x, w, OFF, act)
    else:
        got, _ = products.linear_backward(g, products.linear(x, w, bias, None, OFF, act)[0]["z"][0], x, w, OFF, act)
    h = 1e-6
    for name, v in (("dx", x), ("dw", w), ("dbias", bias)):
        if name not in got:
            continue
        for i in np.ndindex(v.shape):
            old = v[i]
            v[i] = old + h
            up = loss(x, w, bias)
            v[i] = old - h
            down = loss(x, w, bias)
            v[i] = old
            assert abs((up - down) / (2 * h) - got[name][0][i]) < 1e-7, (name, i)


def test_activations_far_out_and_their_bounds():
    """Values and derivatives stay finite for any finite z, and an fp32 evaluation is inside the bounds."""
    z = np.concatenate([np.linspace(-60, 60, 4001), [1e4, -1e4, 1e19, -1e19, 0.0, -0.0]]).astype(np.float32)
    for act in ("silu", "gelu"):
        with np.errstate(all="ignore"):
            v, g, ev, eg = products.activation(z[:4001], act)
            assert np.isfinite(v).all() and np.isfinite(g).all()
            t = torch.from_numpy(z[:4001]).requires_grad_()
            y = torch_act(t, act)
            y.sum().backward()
            assert (np.abs(y.detach().numpy() - v) <= ev + 1e-6 * np.abs(v) + 1e-6).all()
        assert np.abs(g).max() <= products.SLOPE


def test_ranges_bring_entries_into_the_rows():
    assert products.ranges([-5, 2, 9, 4], 6) == [(0, 2), (2, 6), (6, 6)]
    assert products.ranges(None, 6) == [(0, 6)]
