"""fp64 CPU oracle of the operators around the LM head: token sampling and gradient
clipping. Numpy only, written from the formulas of include/lce.h."""
from __future__ import annotations

import numpy as np


def _row(value, i):
    """Setting of row i as the 64-bit value of its 32-bit float."""
    v = np.asarray(value)
    return float(np.float32(v[i] if v.ndim else v))


def sample(Z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Z [N, V] fp64, u [N] -> dict of tokens [N] int64, logprobs [N], and the two parts x
    (distance of the token's logit from the largest over the temperature) and ls (log of
    the kept weight) of logprob = -x - ls."""
    Z = np.asarray(Z, np.float64)
    N, _ = Z.shape
    out = {"tokens": np.full(N, -1, np.int64), "logprobs": np.full(N, -np.inf), "x": np.zeros(N),
           "ls": np.zeros(N), "kept": np.zeros(N, np.int64)}
    for i in range(N):
        z = np.where(np.isnan(Z[i]), -np.inf, Z[i])
        order = np.argsort(-z, kind="stable")
        order = order[z[order] > -np.inf]
        if not order.size:
            continue
        T, k, p, q = (_row(a, i) for a in (temperature, top_k, top_p, min_p))
        if not T > 0:
            out["tokens"][i], out["logprobs"][i], out["kept"][i] = order[0], 0.0, 1
            continue
        with np.errstate(invalid="ignore"):
            x = np.where(z[order] == z[order[0]], 0.0, (z[order[0]] - z[order]) / T)
        if k > 0:
            order, x = order[:int(k)], x[:int(k)]
        w = np.exp(-x)
        keep = np.ones(order.size, bool)
        if p < 1.0:
            keep &= (np.cumsum(w) - w) < p * w.sum()
        if q > 0.0:
            keep &= w >= min(q, 1.0)
        n = max(1, int(keep.sum()))            # a prefix of the order
        order, x, w = order[:n], x[:n], w[:n]
        by_index = np.argsort(order)
        c = np.cumsum(w[by_index])
        j = int(np.searchsorted(c, float(u[i]) * c[-1], side="right"))
        j = min(j, int(np.searchsorted(c, c[-1], side="left")))
        t = by_index[j]
        out["tokens"][i], out["x"][i], out["ls"][i], out["kept"][i] = order[t], x[t], np.log(c[-1]), n
        out["logprobs"][i] = -x[t] - np.log(c[-1])
    return out


def grad_norm(grads, norm_type=2.0):
    """Norm over all values of a list of arrays."""
    flat = [np.asarray(g, np.float64).reshape(-1) for g in grads]
    if norm_type == np.inf:
        return max((np.abs(f).max() if f.size else 0.0) for f in flat)
    if norm_type == 1:
        return sum(np.abs(f).sum() for f in flat)
    return float(np.sqrt(sum((f * f).sum() for f in flat)))


def clip(grads, max_norm, norm_type=2.0, eps=1e-6):
    """(norm, scaled gradients)."""
    norm = grad_norm(grads, norm_type)
    f = min(1.0, max_norm / (norm + eps))
    return norm, [np.asarray(g, np.float64) * f for g in grads]
