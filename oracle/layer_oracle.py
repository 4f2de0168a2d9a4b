"""Plain fp64 implementations of the operators around the expert FFN: the norms
before and after it, the router projection, the low-rank adapters. Straight from
the formulas, one row at a time; shares no code with the GPU path."""
from __future__ import annotations

import numpy as np


def rms_norm(v: np.ndarray, weight: np.ndarray, eps: float) -> np.ndarray:
    """v[t] / sqrt(mean(v[t]^2) + eps) * weight."""
    v = np.asarray(v, np.float64)
    out = np.zeros_like(v)
    for t in range(v.shape[0]):
        out[t] = v[t] / np.sqrt(np.sum(v[t] * v[t]) / v.shape[1] + eps) * weight
    return out


def norm_in(x, weight, residual=None, alpha=1.0, eps=1e-6):
    """(out, s): s = residual + alpha * x, out = rms_norm(s)."""
    s = np.float64(alpha) * np.asarray(x, np.float64)
    if residual is not None:
        s = np.asarray(residual, np.float64) + s
    return rms_norm(s, np.asarray(weight, np.float64), eps), s


def norm_out(y, weights=None, ids=None, E=0, shared=None, gate=None, residual=None, weight=None,
             next_weight=None, scale=1.0, eps=1e-6):
    """(out, next or None) of [T*k, H] expert outputs; a slot whose id is outside
    [0, E) is left out, whatever its row holds."""
    y = np.asarray(y, np.float64)
    T = y.shape[0] if weights is None else weights.shape[0]
    k = y.shape[0] // T if T else 1
    H = y.shape[1]
    out = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            if ids is not None and not 0 <= ids[t, j] < E:
                continue
            w = 1.0 if weights is None else np.float64(weights[t, j])
            out[t] += w * y[t * k + j]
        if shared is not None:
            g = 1.0
            if gate is not None:
                with np.errstate(over="ignore"):
                    g = 1.0 / (1.0 + np.exp(-np.float64(gate[t])))
            out[t] += g * np.asarray(shared[t], np.float64)
    if weight is not None:
        out = rms_norm(out, np.asarray(weight, np.float64), eps)
    out = np.float64(scale) * out
    if residual is not None:
        out = np.asarray(residual, np.float64) + out
    if next_weight is None:
        return out, None
    return out, rms_norm(out, np.asarray(next_weight, np.float64), eps)


def router_logits(x, w, bias=None):
    out = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    return out if bias is None else out + np.asarray(bias, np.float64)


def lora_add(y, x, a, b, ids, scale=None):
    """y[s] + scale[g] * b[g] (a[g] x[s]) for the rows with g = ids[s] in [0, n);
    the other rows are y's."""
    out = np.asarray(y, np.float64).copy()
    n = a.shape[0]
    for g in sorted(set(int(i) for i in ids)):
        if 0 <= g < n:
            rows = np.nonzero(np.asarray(ids) == g)[0]
            z = np.asarray(x[rows], np.float64) @ np.asarray(a[g], np.float64).T
            d = z @ np.asarray(b[g], np.float64).T
            out[rows] += d * (1.0 if scale is None else np.float64(scale[g]))
    return out
