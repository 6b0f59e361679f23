"""Tokens sorted by expert, moved, weighted and brought back; their gradients; the gates' gradient.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The definitions in fp64, pair by pair, with pairs p = t*k + j and a pair kept when its expert id
is in [0, E).  The pages say nothing of gradients; the formulas are the derivatives of these
forward definitions, pinned against differences and against autograd in fp64.
"""
import numpy as np


def sort_pairs(idx, n_experts):
    """(perm of the kept pairs, inv [T,k], offsets [E+1]): stable by (expert, pair)."""
    idx = np.asarray(idx)
    flat = idx.reshape(-1)
    kept = [p for p in range(flat.size) if 0 <= flat[p] < n_experts]
    perm = sorted(kept, key=lambda p: (flat[p], p))
    inv = np.full(flat.size, -1, np.int32)
    for i, p in enumerate(perm):
        inv[p] = i
    offsets = np.array([sum(1 for p in kept if flat[p] < e) for e in range(n_experts + 1)], np.int32)
    return np.array(perm, np.int32), inv.reshape(idx.shape), offsets


def dispatch(x, perm, k):
    """xs[i] = x[perm[i] // k]."""
    return np.asarray(x)[np.asarray(perm, np.int64) // k]


def gather_sum(rows, inv, w=None):
    """(y, s): y[t] = sum_j w[t,j] rows[inv[t,j]] over kept pairs, and s the same sum of magnitudes."""
    rows = np.asarray(rows, np.float64)
    inv = np.asarray(inv)
    T, k = inv.shape
    y, s = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= inv[t, j] < T * k:
                v = rows[inv[t, j]] * (1.0 if w is None else float(w[t, j]))
                y[t] += v
                s[t] += np.abs(v)
    return y, s


def combine_backward(dy, ys, inv, w):
    """(dys, written, dw, s): dys[inv[t,j]] = w[t,j] dy[t], dw[t,j] = <dy[t], ys[inv[t,j]]>; written marks
    the rows that have a pair, s is dw's sum of magnitudes."""
    dy, ys, inv = np.asarray(dy, np.float64), np.asarray(ys, np.float64), np.asarray(inv)
    T, k = inv.shape
    dys, written = np.zeros_like(ys), np.zeros(ys.shape[0], bool)
    dw, s = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            i = inv[t, j]
            if 0 <= i < T * k:
                dys[i] = float(w[t, j]) * dy[t]
                written[i] = True
                dw[t, j] = np.sum(dy[t] * ys[i])
                s[t, j] = np.sum(np.abs(dy[t] * ys[i]))
    return dys, written, dw, s


def topk_gates(z, idx, renorm):
    """The gates of kept pairs as a function of the logits, the choice held (0 for a pair left out)."""
    z, idx = np.asarray(z, np.float64), np.asarray(idx)
    T, E = z.shape
    w = np.zeros(idx.shape)
    for t in range(T):
        kept = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E]
        base = z[t, idx[t, kept]] if renorm else z[t]
        if not kept or np.max(base) == -np.inf:
            continue
        m = np.max(base)
        w[t, kept] = np.exp(z[t, idx[t, kept]] - m) / np.sum(np.exp(base - m))
    return w


def topk_backward(z, idx, dw, renorm):
    """(dz, p, dsum): the gates' gradient and, for error bounds, the softmax values it ran over and the
    sums of |dw| per logit."""
    z, idx, dw = np.asarray(z, np.float64), np.asarray(idx), np.asarray(dw, np.float64)
    T, E = z.shape
    w = topk_gates(z, idx, renorm)
    dz, p, mag = np.zeros((T, E)), np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        if not renorm and np.max(z[t]) > -np.inf:
            p[t] = np.exp(z[t] - np.max(z[t])) / np.sum(np.exp(z[t] - np.max(z[t])))
        mean = 0.0
        for j in range(idx.shape[1]):
            if 0 <= idx[t, j] < E:
                mean += w[t, j] * dw[t, j]
        for j in range(idx.shape[1]):
            e = idx[t, j]
            if 0 <= e < E:
                mag[t, e] += abs(dw[t, j])
                dz[t, e] += w[t, j] * dw[t, j] - (w[t, j] * mean if renorm else 0.0)
                if renorm:
                    p[t, e] = w[t, j]
        if not renorm:
            dz[t] -= p[t] * mean
    return dz, p, mag
