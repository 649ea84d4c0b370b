"""fp64 CPU oracle of the operators around the LM head: token sampling, gradient clipping
and 8-bit quantisation. Numpy only, written from the formulas of include/lce.h."""
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


def e4m3(y):
    """The nearest e4m3 value (ties to even) of each |y| <= 448: 3 bits behind the leading
    one, exponents -6 to 8, steps of 2^-9 below. NaN and infinities: NaN."""
    y = np.asarray(y, np.float64)
    ok = np.isfinite(y)
    a = np.where(ok, np.abs(y), 0.0)
    _, e = np.frexp(a)                                  # a = f 2^e, f in [0.5, 1)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    r = np.round(a / step) * step                       # numpy rounds ties to even
    return np.where(ok, np.copysign(r, y), np.nan)


def quantize_fp8(X, tiles=False):
    """(values q, scale) of X [R, C] fp64 in row blocks of 128 or tiles of 128 x 128."""
    X = np.asarray(X, np.float64)
    R, C = X.shape
    rows = 128 if tiles else 1
    RB, CB = -(-R // rows), -(-C // 128)
    P = np.zeros((RB * rows, CB * 128))
    P[:R, :C] = X
    T = P.reshape(RB, rows, CB, 128)
    amax = np.where(np.isfinite(T), np.abs(T), 0.0).max(axis=(1, 3))
    f, e = np.frexp(amax)                               # 448 = 0.875 * 2^9
    e = np.maximum(e - 9 + (f > 0.875), -126)
    scale = np.where(amax > 0, np.ldexp(1.0, e), 1.0)
    q = e4m3(T / scale[:, None, :, None])
    return q.reshape(P.shape)[:R, :C], scale


def dequantize_fp8(q, scale):
    """Values of an operand: scale [R, CB] or [ceil(R / 128), CB]."""
    q = np.asarray(q, np.float64)
    R, C = q.shape
    s = np.repeat(np.asarray(scale, np.float64), 128, axis=1)[:, :C]
    return q * (s if s.shape[0] == R else np.repeat(s, 128, axis=0)[:R])
