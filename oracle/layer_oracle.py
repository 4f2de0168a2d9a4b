"""Plain fp64 implementations of the operators around the expert FFN: the norms
before and after it, the router projection, the low-rank adapters; and of those
beside it: tokens in expert order and back, layer norm, the product with an
epilogue. Straight from the formulas, one row at a time; shares no code with the
GPU path."""
from __future__ import annotations

import math

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


def places(sorted_ids, num_padded, S):
    """Every slot's place in the lists of an alignment, -1 for none."""
    at = np.full(S, -1, np.int64)
    for p in range(int(num_padded)):
        if 0 <= sorted_ids[p] < S:
            at[sorted_ids[p]] = p
    return at


def dispatch(x, sorted_ids, num_padded, k):
    """rows [num_padded, H]: each slot's token at its place, zeros in the padding."""
    x = np.asarray(x)
    rows = np.zeros((int(num_padded), x.shape[1]), x.dtype)
    for p in range(int(num_padded)):
        if 0 <= sorted_ids[p] < x.shape[0] * k:
            rows[p] = x[sorted_ids[p] // k]
    return rows


def combine(rows, at, weights=None):
    """out[t] = sum_j weights[t, j] rows[at[t, j]] over the slots with a place."""
    T, k = at.shape
    out = np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= at[t, j] < rows.shape[0]:
                w = 1.0 if weights is None else np.float64(weights[t, j])
                out[t] += w * np.asarray(rows[at[t, j]], np.float64)
    return out


def combine_backward(dout, rows, at, weights, num_padded):
    """(drows [num_padded, H], dweights [T, k])."""
    T, k = at.shape
    drows = np.zeros((int(num_padded), rows.shape[1]))
    dweights = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if 0 <= at[t, j] < rows.shape[0]:
                w = 1.0 if weights is None else np.float64(weights[t, j])
                drows[at[t, j]] = w * dout[t]
                dweights[t, j] = np.sum(np.asarray(dout[t], np.float64) * rows[at[t, j]])
    return drows, dweights


def layer_norm(x, weight=None, bias=None, residual=None, alpha=1.0, eps=1e-5):
    """(out, s): s = residual + alpha * x, out = (s - mean) / sqrt(var + eps) * weight + bias."""
    s = np.float64(alpha) * np.asarray(x, np.float64)
    if residual is not None:
        s = np.asarray(residual, np.float64) + s
    out = np.zeros_like(s)
    for t in range(s.shape[0]):
        d = s[t] - np.sum(s[t]) / s.shape[1]
        out[t] = d / np.sqrt(np.sum(d * d) / s.shape[1] + eps)
    if weight is not None:
        out = out * np.asarray(weight, np.float64)
    return out if bias is None else out + np.asarray(bias, np.float64), s


def layer_norm_backward(dout, s, weight=None, dresidual_out=None, alpha=1.0, eps=1e-5):
    """(dx, ds, dweight, dbias) of layer_norm at the sum s."""
    dout, s = np.asarray(dout, np.float64), np.asarray(s, np.float64)
    T, H = s.shape
    w = np.ones(H) if weight is None else np.asarray(weight, np.float64)
    ds, dweight, dbias = np.zeros_like(s), np.zeros(H), np.zeros(H)
    for t in range(T):
        d = s[t] - np.sum(s[t]) / H
        inv = 1.0 / np.sqrt(np.sum(d * d) / H + eps)
        u, g = d * inv, dout[t] * w
        ds[t] = inv * (g - np.sum(g) / H - u * np.sum(g * u) / H)
        dweight += dout[t] * u
        dbias += dout[t]
    if dresidual_out is not None:
        ds = ds + np.asarray(dresidual_out, np.float64)
    return np.float64(alpha) * ds, ds, dweight, dbias


def activate(name, v):
    """none, relu, silu, gelu (by erf) or gelu_tanh."""
    v = np.asarray(v, np.float64)
    if name == "relu":
        return np.maximum(v, 0.0)
    if name == "silu":
        with np.errstate(over="ignore"):
            return v / (1.0 + np.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1.0 + np.vectorize(math.erf, otypes=[float])(v / math.sqrt(2.0)))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    assert name == "none"
    return v


def linear(x, w, bias=None, act="none", gated=False, residual=None):
    """residual + act(x w^T + bias); gated: w holds gate rows, then as many up rows."""
    v = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    if bias is not None:
        v = v + np.asarray(bias, np.float64)
    if gated:
        N = v.shape[1] // 2
        v = activate(act, v[:, :N]) * v[:, N:]
    else:
        v = activate(act, v)
    return v if residual is None else np.asarray(residual, np.float64) + v
