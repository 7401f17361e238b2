"""Float64 log probabilities of given tokens and distillation from a teacher's largest logits."""
import numpy as np


def log_softmax(l, temperature):
    """(u - max u, log p, p) of rows of logits; a row of -inf has log p -inf and p 0."""
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        m = l.max(1, keepdims=True)
        d = np.where(m == -np.inf, -np.inf, (l - np.where(np.isfinite(m), m, 0.0)) / temperature)
        s = np.log(np.exp(d).sum(1, keepdims=True))
        lp = np.where(m == -np.inf, -np.inf, d - s)
    return d, lp, np.exp(lp)


def plogp(p, lp):
    with np.errstate(invalid="ignore"):
        return np.where(p > 0, p * lp, 0.0)


def logprobs(l, targets, top, temperature):
    """dict: logprob, entropy, top_ids, top_logprobs, and d, lp, p of the rows."""
    T, V = l.shape
    d, lp, p = log_softmax(l, temperature)
    has = (targets >= 0) & (targets < V)
    logprob = np.where(has, lp[np.arange(T), np.where(has, targets, 0)], 0.0)
    ids = np.argsort(-l, axis=1, kind="stable")[:, :top]
    return {"logprob": logprob, "entropy": -plogp(p, lp).sum(1), "top_ids": ids,
            "top_logprobs": np.take_along_axis(lp, ids, 1), "d": d, "lp": lp, "p": p, "has": has}


def logprobs_grad(r, targets, g, h, temperature):
    p, lp = r["p"], r["lp"]
    y = np.zeros_like(p)
    y[np.nonzero(r["has"])[0], targets[r["has"]]] = 1.0
    return ((g * r["has"])[:, None] * (y - p) - h[:, None] * (plogp(p, lp) + p * r["entropy"][:, None])) / temperature


def teacher(V, ids, values, temperature, lse):
    """(q, ln q) of the rows' entries, 0 and -inf where there is none."""
    there = (ids >= 0) & (ids < V)
    with np.errstate(invalid="ignore", divide="ignore"):
        v = np.where(there, values / temperature, -np.inf)
        if lse is None:
            m = v.max(1, keepdims=True)
            m = np.where(np.isfinite(m), m, 0.0)
            lnq = v - m - np.log(np.exp(v - m).sum(1, keepdims=True))
        else:
            lnq = v - lse[:, None]
        lnq = np.where(v == -np.inf, -np.inf, lnq)
    return np.exp(lnq), lnq


def distill(l, ids, values, g, temperature=1.0, mask=None, lse=None):
    """(loss, gradient, q, ln q, and d, log p, p of the rows)."""
    T, V = l.shape
    keep = np.ones(T, bool) if mask is None else mask.astype(bool)
    d, lp, p = log_softmax(np.where(keep[:, None], l, 0.0), temperature)
    q, lnq = teacher(V, ids, values, temperature, lse)
    at = np.where(q > 0, ids, 0)
    with np.errstate(invalid="ignore"):
        term = np.where(q > 0, q * (lnq - np.take_along_axis(lp, at, 1)), 0.0)
    grad = q.sum(1, keepdims=True) * p
    for t in range(T):
        np.add.at(grad[t], at[t], -q[t])
    grad *= (g * keep / temperature)[:, None]
    return term.sum(1) * keep, grad, q, lnq, d, lp, p
