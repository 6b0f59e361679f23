"""The experts' products over rows sorted by expert, and their gradients.

TEST INFRASTRUCTURE ONLY (see the package docstring).

glu:     gu = x w^T (gate columns, then up), a = act(gate) up
linear:  z = x w^T + b, y = act(z) + r
with silu(z) = z s(z), gelu in its tanh form, s the logistic function, expert by expert in fp64.  The
pages say nothing of these; gradients are the derivatives of the definitions, pinned against
differences.

Beside each result stands a bound on an evaluation in fp32 with operands as given.  A sum of n
products whose every addition and product errs by at most one step (2^-23 of its value, rounded or cut)
errs by at most (n + 8) 2^-23 times the sum of magnitudes.  A logistic function at q, by an
exponential, an addition and a quotient, with q itself off by 8 half steps, errs by (16 + 8 |q|) 2^-24 of its
value.  d, the gradient before a projection, becomes an operand of its type: off by `u_op` (half a
step, relative) more.
"""
import numpy as np

STEP = 2.0 ** -23
SLOPE = 1.2   # no activation here is steeper: silu 1.0998, gelu 1.129


def _logistic(q):
    return 0.5 * (1.0 + np.tanh(0.5 * q))


def _inner(z, act):
    """(q, dq/dz) of the activation z s(q)."""
    if act == "silu":
        return z, np.ones_like(z)
    c = 2.0 * np.sqrt(2.0 / np.pi)
    return c * (z + 0.044715 * z ** 3), c * (1.0 + 3 * 0.044715 * z ** 2)


def activation(z, act):
    """(value, derivative, bound of the value's error, bound of the derivative's)."""
    z = np.asarray(z, np.float64)
    if act == "none":
        return z, np.ones_like(z), np.zeros_like(z), np.zeros_like(z)
    q, dq = _inner(z, act)
    s, c = _logistic(q), _logistic(-q)
    rel = (16.0 + 8.0 * np.minimum(np.abs(q), 200.0)) * STEP / 2
    return z * s, s + z * s * c * dq, rel * np.abs(z * s) + 1e-38, 2 * rel * (s + np.abs(z * dq) * s * c) + 1e-38


def ranges(offsets, rows):
    """[(first, end)] of each expert's rows; offsets None: one expert of all."""
    if offsets is None:
        return [(0, rows)]
    off = np.clip(np.asarray(offsets, np.int64), 0, rows)
    return [(int(a), int(max(a, b))) for a, b in zip(off[:-1], off[1:])]


def _product(x, w):
    """x w^T and its error's bound."""
    return x @ w.T, (x.shape[1] + 8) * STEP * (np.abs(x) @ np.abs(w).T)


def glu(x, w, offsets, act):
    """{name: (value, bound)} of a and gu, and the rows that have an expert."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    R, N = x.shape[0], w.shape[1]
    I = N // 2
    out = {k: (np.zeros((R, n)), np.zeros((R, n))) for k, n in (("a", I), ("gu", N))}
    kept = np.zeros(R, bool)
    for e, (lo, hi) in enumerate(ranges(offsets, R)):
        gu, err = _product(x[lo:hi], w[e])
        v, _, ev, _ = activation(gu[:, :I], act)
        u = gu[:, I:]
        out["gu"][0][lo:hi], out["gu"][1][lo:hi] = gu, err
        out["a"][0][lo:hi] = v * u
        dv = SLOPE * err[:, :I] + ev
        out["a"][1][lo:hi] = dv * (np.abs(u) + err[:, I:]) + np.abs(v) * err[:, I:] + STEP * np.abs(v * u)
        kept[lo:hi] = True
    return out, kept


def linear(x, w, bias, residual, offsets, act):
    """The same of z and y."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    R, N = x.shape[0], w.shape[1]
    out = {k: (np.zeros((R, N)), np.zeros((R, N))) for k in ("z", "y")}
    kept = np.zeros(R, bool)
    for e, (lo, hi) in enumerate(ranges(offsets, R)):
        z, err = _product(x[lo:hi], w[e])
        if bias is not None:
            z = z + np.asarray(bias, np.float64)[e]
            err = err + STEP * np.abs(z)
        y, _, ev, _ = activation(z, act)
        ey = (SLOPE if act != "none" else 1.0) * err + ev
        if residual is not None:
            y = y + np.asarray(residual, np.float64)[lo:hi]
            ey = ey + STEP * np.abs(y)
        out["z"][0][lo:hi], out["z"][1][lo:hi] = z, err
        out["y"][0][lo:hi], out["y"][1][lo:hi] = y, ey
        kept[lo:hi] = True
    return out, kept


def _gradients(d, ed, x, w, offsets, u_op):
    """dx, dw of the gradient d before the projection, off by ed and by its rounding as an operand."""
    d, w, x = np.asarray(d, np.float64), np.asarray(w, np.float64), np.asarray(x, np.float64)
    ed = ed + u_op * (np.abs(d) + ed) + 1e-38
    R = d.shape[0]
    out = {"dx": (np.zeros_like(x), np.zeros_like(x)), "dw": (np.zeros_like(w), np.zeros_like(w))}
    kept = np.zeros(R, bool)
    for e, (lo, hi) in enumerate(ranges(offsets, R)):
        de, ee, xe = d[lo:hi], ed[lo:hi], x[lo:hi]
        aw, mag = np.abs(w[e]), np.abs(de) + ee
        out["dx"][0][lo:hi] = de @ w[e]
        out["dx"][1][lo:hi] = ee @ aw + (w.shape[1] + 8) * STEP * (mag @ aw)
        out["dw"][0][e] = de.T @ xe
        out["dw"][1][e] = ee.T @ np.abs(xe) + (hi - lo + 8) * STEP * (mag.T @ np.abs(xe))
        kept[lo:hi] = True
    return out, kept


def glu_backward(da, gu, x, w, offsets, act, u_op=0.0):
    da, gu = np.asarray(da, np.float64), np.asarray(gu, np.float64)
    I = da.shape[1]
    u = gu[:, I:]
    v, g, ev, eg = activation(gu[:, :I], act)
    d = np.concatenate([da * u * g, da * v], axis=1)
    ed = np.concatenate([np.abs(da * u) * eg, np.abs(da) * ev], axis=1) + 2 * STEP * np.abs(d)
    return _gradients(d, ed, x, w, offsets, u_op)


def linear_backward(dy, z, x, w, offsets, act, u_op=0.0):
    """Also dbias, whose terms are not rounded as operands."""
    dy = np.asarray(dy, np.float64)
    if act == "none":
        d, ed = dy, np.zeros_like(dy)
    else:
        _, g, _, eg = activation(z, act)
        d = dy * g
        ed = np.abs(dy) * eg + STEP * np.abs(d)
    out, kept = _gradients(d, ed, x, w, offsets, u_op)
    rs = ranges(offsets, dy.shape[0])
    out["dbias"] = (np.stack([d[lo:hi].sum(0) for lo, hi in rs]),
                    np.stack([(ed[lo:hi] + (hi - lo + 8) * STEP * np.abs(d[lo:hi])).sum(0) for lo, hi in rs]))
    return out, kept
