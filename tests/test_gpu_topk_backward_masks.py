"""GPU: the gates' gradient where a masked or unchosen logit meets a gradient that is infinite or NaN:
what has no share gets exactly 0 and adds nothing."""
import numpy as np
import pytest
import torch

from oracle import tokens
from test_gpu_tokens import F, R, U32, dev, within

pytestmark = pytest.mark.gpu

INF, NAN = np.inf, np.nan


def run(z, idx, dw, renorm):
    z, idx, dw = np.asarray(z, np.float32), np.asarray(idx, np.int32), np.asarray(dw, np.float32)
    got = torch.full(z.shape, 9.0, device="cuda")
    R().moe_topk_backward(dev(z), dev(idx), dev(dw), renorm, got)
    return got


@pytest.mark.parametrize("bad", [INF, -INF, NAN])
@pytest.mark.parametrize("E,k", [(3, 2), (8, 3), (257, 5), (1000, 70)])
@pytest.mark.parametrize("renorm", [0, 1])
def test_pairs_at_masked_logits_add_nothing(E, k, renorm, bad):
    """Against the definition with those pairs' gradients 0."""
    T = 9
    rng = np.random.default_rng(E + k)
    z = rng.standard_normal((T, E))
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    dw = rng.standard_normal((T, k))
    clean = dw.copy()
    for t in range(T):
        z[t, idx[t, t % k]] = -INF
        dw[t, t % k], clean[t, t % k] = bad, 0.0
    z = z.astype(np.float32)
    clean = clean.astype(np.float32)
    got = run(z, idx, dw, renorm)
    ref, p, mag = tokens.topk_backward(z, idx, clean, renorm)
    # as in the test of finite gradients: logits within 10 of each other
    rel = 2 * (2 * 10 + 8 + E / 64 + 8) * U32
    M = np.sum(p * mag, axis=1, keepdims=True)
    within(got, ref, p * (mag + M) * (2 * rel + (k + 24) * U32), F)
    assert all(got[t, idx[t, t % k]] == 0 for t in range(T))


@pytest.mark.parametrize("bad", [INF, NAN, 1.0])
@pytest.mark.parametrize("renorm", [0, 1])
def test_every_logit_masked(renorm, bad):
    z = np.full((5, 12), -INF)
    got = run(z, np.arange(10).reshape(5, 2), np.full((5, 2), bad), renorm)
    assert (got == 0).all()


@pytest.mark.parametrize("bad", [INF, NAN])
def test_unchosen_stay_zero_with_renorm(bad):
    """A gradient that is not finite belongs to the chosen experts of its token alone."""
    z = np.zeros((3, 16))
    idx = np.array([[1, 5], [2, 3], [15, 0]])
    dw = np.ones((3, 2))
    dw[1, 0] = bad
    got = run(z, idx, dw, 1).cpu()
    chosen = torch.zeros(3, 16, dtype=torch.bool).scatter_(1, torch.from_numpy(idx), True)
    assert (got[~chosen] == 0).all()
    assert got[1, 2].isnan() and not got[[0, 2]].isnan().any()


def test_nan_logits_are_not_hidden():
    """Nor are infinite ones (inf - inf): the token's gradients are NaN, but for masked logits."""
    z = np.zeros((3, 6))
    z[0, 4], z[2, 4] = NAN, INF
    z[0, 5] = z[2, 5] = -INF
    got = run(z, [[0, 1]] * 3, np.ones((3, 2)), 0)
    assert got[[0, 2], :5].isnan().all() and got[1].isfinite().all() and (got[[0, 2], 5] == 0).all()
