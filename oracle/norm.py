"""The norms before and after a block, with its gate and residual scale, and their gradient.

TEST INFRASTRUCTURE ONLY (see the package docstring).

rms(v) = sqrt(mean(v^2) + eps) over a row.  The pages give the layer's inside only; the step
between two layers is the plain pre-norm / post-norm transformer block with RMS norms.  Pinned
against differences and autograd in fp64.
"""
import numpy as np


def _col(gate, T, per_token):
    if gate is None:
        return np.ones((T, 1))
    gate = np.asarray(gate, np.float64)
    return gate[:, None] if per_token else gate[None, :]


def _rms(v, eps):
    return np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)


def block_norm(h, y, w_post, gate, per_token, w_pre, alpha, eps):
    """(h_out, x_out or None)."""
    h = np.asarray(h, np.float64)
    if y is not None:
        y = np.asarray(y, np.float64)
        u = y if w_post is None else np.asarray(w_post, np.float64) * y / _rms(y, eps)
        h = h + alpha * _col(gate, h.shape[0], per_token) * u
    return h, None if w_pre is None else np.asarray(w_pre, np.float64) * h / _rms(h, eps)


def block_norm_backward(h_out, y, w_post, gate, per_token, w_pre, dh_out, dx, alpha, eps, depth=0, step=0.0):
    """Gradients and, beside each, a bound on an fp32 evaluation's error: {name: (value, bound)}.

    step is half a unit in the last place of fp32 (2^-24), depth how many roundings a row's sum can
    pass through; a sum of n terms with each partial rounded errs by at most depth * step times
    the sum of magnitudes, and errors of dh enter dy and the weights' gradients to first order.
    """
    some = dh_out if dh_out is not None else dx
    T, H = np.asarray(some).shape
    zero = np.zeros((T, H))
    out = {}
    dh = zero if dh_out is None else np.asarray(dh_out, np.float64)
    e = (depth + 16) * step
    edh = e * np.abs(dh)
    if dx is not None:
        hv, dx, wp = np.asarray(h_out, np.float64), np.asarray(dx, np.float64), np.asarray(w_pre, np.float64)
        r = 1.0 / _rms(hv, eps)
        d = wp * dx
        dh = dh + r * (d - hv * r ** 2 * np.mean(d * hv, axis=1, keepdims=True))
        edh = edh + e * r * (np.abs(d) + np.abs(hv) * r ** 2 * np.mean(np.abs(d * hv), axis=1, keepdims=True))
        out["dw_pre"] = (np.sum(dx * hv * r, axis=0), (e + (T + 32) * step) * np.sum(np.abs(dx * hv * r), axis=0))
    out["dh"] = (dh, edh)
    if y is None:
        return out
    y = np.asarray(y, np.float64)
    g = alpha * _col(gate, T, per_token)
    wq = np.ones(H) if w_post is None else np.asarray(w_post, np.float64)
    du, edu = g * dh, np.abs(g) * (edh + 4 * step * np.abs(dh))
    es = (T + 32) * step
    if w_post is None:
        u, ry = y, np.ones((T, 1))
        out["dy"] = (du, edu)
    else:
        ry = 1.0 / _rms(y, eps)
        u = wq * y * ry
        mean = lambda v: np.mean(v, axis=1, keepdims=True)  # noqa: E731
        out["dy"] = (ry * (wq * du - y * ry ** 2 * mean(wq * du * y)),
                     ry * (np.abs(wq) * edu + np.abs(y) * ry ** 2 * mean(np.abs(wq * y) * edu))
                     + e * ry * (np.abs(wq * du) + np.abs(y) * ry ** 2 * mean(np.abs(wq * du * y))))
        out["dw_post"] = (np.sum(du * y * ry, axis=0),
                          np.sum(np.abs(y * ry) * edu + (e + es) * np.abs(du * y * ry), axis=0))
    if gate is not None:
        axis = 1 if per_token else 0
        v = alpha * dh * u
        out["dgate"] = (np.sum(v, axis=axis), np.sum(abs(alpha) * edh * np.abs(u) + (e + es) * np.abs(v), axis=axis))
    return out
