"""Float64 products by expert with 16-bit weights, and both gradients."""
import numpy as np


def sources(ids, per_route):
    """Row of x that each route reads."""
    T, k = ids.shape
    return np.arange(T * k) if per_route else np.arange(T * k) // k


def plan(ids, E):
    """Routes by expert (ascending within one, those of no expert last) and the groups' beginnings."""
    flat = ids.reshape(-1).astype(np.int64)
    group = np.where((flat >= 0) & (flat < E), flat, E)
    counts = np.bincount(group, minlength=E + 1)
    return np.argsort(group, kind="stable"), np.concatenate([[0], np.cumsum(counts)[:E]])


def forward(x, w, ids, per_route):
    """(rows [T * k, N], sums of the products' magnitudes)."""
    src, flat = sources(ids, per_route), ids.reshape(-1)
    y = np.zeros((flat.size, w.shape[1]))
    mag = np.zeros_like(y)
    for r, e in enumerate(flat):
        if 0 <= e < w.shape[0]:
            y[r] = w[e] @ x[src[r]]
            mag[r] = np.abs(w[e]) @ np.abs(x[src[r]])
    return y, mag


def backward(x, w, ids, grad_out, per_route):
    """(grad_x, grad_w, and for each the sums of the products' magnitudes)."""
    src, flat = sources(ids, per_route), ids.reshape(-1)
    gx, gw = np.zeros(x.shape), np.zeros(w.shape)
    mx, mw = np.zeros(x.shape), np.zeros(w.shape)
    for r, e in enumerate(flat):
        if 0 <= e < w.shape[0]:
            gx[src[r]] += grad_out[r] @ w[e]
            mx[src[r]] += np.abs(grad_out[r]) @ np.abs(w[e])
            gw[e] += np.outer(grad_out[r], x[src[r]])
            mw[e] += np.abs(np.outer(grad_out[r], x[src[r]]))
    return gx, gw, mx, mw
