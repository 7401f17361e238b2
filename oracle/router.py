"""Router with load statistics, losses and its gradient (oracle; test use only).

Everything in float64 from the logits' own values; token by token.
"""
from __future__ import annotations

import numpy as np


def forward(logits, k: int, mask=None):
    """dict of ids, w, lse, counts, prob, losses, tokens (see trellis_moe_router_forward)."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    ids = np.zeros((T, k), dtype=np.int64)
    w = np.zeros((T, k))
    lse = np.full(T, -np.inf)
    counts = np.zeros(E, dtype=np.int64)
    prob = np.zeros(E)
    z = 0.0
    n = 0
    for t in range(T):
        order = sorted(range(E), key=lambda e: (-l[t, e], e))
        ids[t] = order[:k]
        m = l[t, order[0]]
        if m == -np.inf:
            continue
        ex = np.exp(l[t] - m)
        lse[t] = m + np.log(ex.sum())
        w[t] = ex[ids[t]] / ex[ids[t]].sum()
        if mask is not None and not mask[t]:
            continue
        n += 1
        prob += ex / ex.sum()
        z += lse[t] ** 2
        for e in ids[t]:
            counts[e] += l[t, e] > -np.inf
    inv = 1.0 / n if n else 0.0
    prob *= inv
    losses = np.array([E * np.sum(counts * inv / k * prob), z * inv])
    return {"ids": ids, "w": w, "lse": lse, "counts": counts, "prob": prob, "losses": losses, "tokens": n}


def loss_of(logits, k: int, mask, grad_w, grad_losses, ids, counts):
    """Scalar whose gradient `backward` states: selections and counts held at `ids` and `counts`."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    valid = [t for t in range(T) if np.max(l[t]) > -np.inf and (mask is None or mask[t])]
    n = len(valid)
    total = 0.0
    if n:
        p = np.exp(l[valid] - l[valid].max(1, keepdims=True))
        s = p.sum(1, keepdims=True)
        lse = np.log(s[:, 0]) + l[valid].max(1)
        prob = (p / s).mean(0)
        total += grad_losses[0] * E * np.sum(counts / (n * k) * prob) + grad_losses[1] * np.mean(lse ** 2)
    for t in range(T):
        if np.max(l[t]) > -np.inf:
            v = np.exp(l[t, ids[t]] - l[t, ids[t]].max())
            total += np.sum(grad_w[t] * v / v.sum())
    return total


def backward(logits, k: int, mask, fwd, grad_w, grad_losses):
    """Gradient [T, E] and, beside it, the sum of the magnitudes of its terms."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    n = fwd["tokens"]
    f = fwd["counts"] / (n * k) if n else np.zeros(E)
    for t in range(T):
        if fwd["lse"][t] == -np.inf:
            continue
        if mask is None or mask[t]:
            p = np.exp(l[t] - l[t].max())       # (not through lse, which 1e30 leaves without its fraction)
            p /= p.sum()
            a, b = grad_losses[0] * E / n, 2 * grad_losses[1] / n * fwd["lse"][t]
            d[t] += p * (a * (f - np.sum(f * p)) + b)
            mag[t] += p * (abs(a) * (f + np.sum(f * p)) + abs(b))
        if grad_w is not None:
            w, g = fwd["w"][t], grad_w[t]
            dot = np.sum(w * g)
            for j, e in enumerate(fwd["ids"][t]):
                d[t, e] += w[j] * (g[j] - dot)
                mag[t, e] += w[j] * (abs(g[j]) + np.sum(np.abs(w * g)))
    return d, mag
