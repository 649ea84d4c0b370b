"""fp64 CPU oracle of the losses on answers (policy, preference) and of the 4-bit linear layer.
Numpy only, written from the formulas of include/lce.h."""
from __future__ import annotations

import numpy as np


def _f64(x):
    return None if x is None else np.asarray(x, np.float64)


def log_softmax_of(Z, y, temperature=1.0, ignore_index=-100):
    """(log p of each counting row's label, else 0; p [N, V], zeros for the other rows; counting)."""
    Z, y = _f64(Z), np.asarray(y)
    N, V = Z.shape
    ok = (y != ignore_index) & (y >= 0) & (y < V)
    p, logp = np.zeros((N, V)), np.zeros(N)
    for i in np.flatnonzero(ok):
        x = Z[i] / temperature
        with np.errstate(invalid="ignore"):
            x = x - x.max()
            e = np.exp(x)
            p[i] = e / e.sum()
            logp[i] = x[y[i]] - np.log(e.sum())
    return logp, p, ok


def _gradient(p, y, ok, scale):
    g = p.copy()
    g[np.flatnonzero(ok), np.asarray(y)[ok]] -= 1.0
    return g * np.where(ok, scale, 0.0)[:, None]


def policy(Z, y, advantages, old=None, ref=None, weights=None, clip_low=0.2, clip_high=0.2, beta=0.0,
           temperature=1.0, reduction="mean", dloss=1.0, ignore_index=-100):
    """dict of loss, logprobs, dZ, and the largest terms of each row's coefficient (mass)."""
    logp, p, ok = log_softmax_of(Z, y, temperature, ignore_index)
    a = _f64(advantages)
    w = np.ones_like(a) if weights is None else _f64(weights)
    r = np.ones_like(a) if old is None else np.exp(logp - _f64(old))
    free, held = r * a, np.clip(r, 1 - clip_low, 1 + clip_high) * a
    loss, slope, mass = -np.minimum(free, held), np.where(free <= held, -free, 0.0), np.abs(free)
    if beta:
        d = _f64(ref) - logp
        loss, slope, mass = loss + beta * (np.expm1(d) - d), slope - beta * np.expm1(d), mass + beta * (1 + np.exp(d))
    rows = np.where(ok, w * loss, 0.0)
    share = np.broadcast_to(_f64(dloss), a.shape) * w
    if reduction == "mean":
        share = share / max(1, ok.sum())
        total = rows.sum() / max(1, ok.sum())
    else:
        total = rows if reduction == "none" else rows.sum()
    scale = -slope * share / temperature
    return {"loss": total, "logprobs": logp, "dZ": _gradient(p, y, ok, scale), "p": p, "ok": ok,
            "mass": np.where(ok, mass * np.abs(share) / temperature, 0.0),
            "terms": np.where(ok, np.abs(w) * (np.abs(loss) + mass), 0.0)}


def preference(Z, y, offsets, ref=None, beta=0.1, smoothing=0.0, average=False, reduction="mean", dloss=1.0,
               ignore_index=-100):
    """dict of loss, seq_logprobs, dZ and coef (what each row's p - onehot is multiplied by)."""
    logp, p, ok = log_softmax_of(Z, y, 1.0, ignore_index)
    S = len(offsets) - 1
    P = S // 2
    parts = [np.arange(offsets[s], offsets[s + 1]) for s in range(S)]
    size = np.array([max(1, int(ok[i].sum())) if average else 1 for i in parts], np.float64)
    seq = np.array([logp[i].sum() for i in parts]) / size
    x = seq - (0.0 if ref is None else _f64(ref))
    m = beta * (x[:P] - x[P:])
    right, wrong = -np.logaddexp(0, -m), -np.logaddexp(0, m)
    rows = -((1 - smoothing) * right + smoothing * wrong)
    d = np.broadcast_to(_f64(dloss), (P,)) / (P if reduction == "mean" else 1)
    slope = beta * (smoothing * np.exp(right) - (1 - smoothing) * np.exp(wrong)) * d
    coef = np.zeros(len(logp))
    for k in range(P):
        coef[parts[k]] = -slope[k] / size[k]
        coef[parts[P + k]] = slope[k] / size[P + k]
    coef = np.where(ok, coef, 0.0)
    loss = rows if reduction == "none" else rows.mean() if reduction == "mean" else rows.sum()
    return {"loss": loss, "seq_logprobs": seq, "dZ": _gradient(p, y, ok, coef), "p": p, "ok": ok, "coef": coef,
            "margin": m}


def int4_values(q, scale, group, D):
    """The weight [V, D] that packed values stand for: (q - 8) * scale of its group."""
    q = np.asarray(q)
    w = np.empty((q.shape[0], 2 * q.shape[1]))
    w[:, 0::2], w[:, 1::2] = q & 15, q >> 4
    return (w[:, :D] - 8.0) * np.repeat(_f64(scale), group, 1)[:, :D]


def quantize_int4(W, group, round_scale):
    """(values -8 .. 7 [V, D], scale [V, groups]): the scale is a seventh of the group's largest
    magnitude, rounded by `round_scale`; 1 for a group of zeros."""
    W = _f64(W)
    V, D = W.shape
    G = -(-D // group)
    x = np.zeros((V, G * group))
    x[:, :D] = W
    x = x.reshape(V, G, group)
    s = round_scale(np.abs(x).max(2) / 7.0)
    s = np.where(s > 0, s, 1.0)
    return np.clip(np.rint(x / s[:, :, None]), -8, 7).reshape(V, -1)[:, :D], s
