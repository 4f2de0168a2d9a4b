"""Pins of the fp64 oracle of the operators around the FFN: brute-force loops on
tiny shapes, closed forms, invariants; and that each pin sees a planted mistake."""
import math

import numpy as np
import pytest

from oracle import layer_oracle as lo


def _rng(seed):
    return np.random.default_rng(seed)


def test_norm_in_brute_force():
    r = _rng(0)
    x, res, w = r.standard_normal((3, 8)), r.standard_normal((3, 8)), r.standard_normal(8)
    out, s = lo.norm_in(x, w, res, alpha=-0.5, eps=1e-3)
    for t in range(3):
        row = [res[t, c] - 0.5 * x[t, c] for c in range(8)]
        inv = 1.0 / math.sqrt(sum(v * v for v in row) / 8 + 1e-3)
        for c in range(8):
            assert math.isclose(s[t, c], row[c], rel_tol=1e-14)
            assert math.isclose(out[t, c], row[c] * inv * w[c], rel_tol=1e-13)


def test_norm_closed_forms():
    # a row of one value v: v / sqrt(v^2 + eps); a zero row stays zero
    out, s = lo.norm_in(np.array([[3.0] * 4, [0.0] * 4]), np.full(4, 2.0), eps=7.0)
    assert np.allclose(out, [[2 * 3 / 4.0] * 4, [0.0] * 4]) and np.array_equal(s[0], [3.0] * 4)
    # scaling a row does not change its norm without eps
    x = _rng(1).standard_normal((2, 16))
    assert np.allclose(lo.norm_in(5 * x, np.ones(16), eps=0.0)[0],
                       lo.norm_in(x, np.ones(16), eps=0.0)[0], rtol=1e-13)


def _norm_out_args(seed=2, T=4, k=3, H=8, E=5):
    r = _rng(seed)
    ids = np.stack([r.permutation(E + 3)[:k] for _ in range(T)])
    return dict(y=r.standard_normal((T * k, H)), weights=r.random((T, k)), ids=ids, E=E,
                shared=r.standard_normal((T, H)), gate=r.standard_normal(T),
                residual=r.standard_normal((T, H)), weight=r.standard_normal(H),
                next_weight=r.standard_normal(H), scale=0.7, eps=1e-2)


def _norm_out_loops(a):
    T, k = a["weights"].shape
    H = a["y"].shape[1]
    outs, nexts = [], []
    for t in range(T):
        v = [0.0] * H
        for j in range(k):
            if 0 <= a["ids"][t, j] < a["E"]:
                for c in range(H):
                    v[c] += a["weights"][t, j] * a["y"][t * k + j, c]
        g = 1 / (1 + math.exp(-a["gate"][t]))
        v = [v[c] + g * a["shared"][t, c] for c in range(H)]
        inv = 1 / math.sqrt(sum(q * q for q in v) / H + a["eps"])
        o = [a["residual"][t, c] + a["scale"] * v[c] * inv * a["weight"][c] for c in range(H)]
        inv = 1 / math.sqrt(sum(q * q for q in o) / H + a["eps"])
        outs.append(o)
        nexts.append([o[c] * inv * a["next_weight"][c] for c in range(H)])
    return np.array(outs), np.array(nexts)


def test_norm_out_brute_force():
    a = _norm_out_args()
    got, ref = lo.norm_out(**a), _norm_out_loops(a)
    assert np.allclose(got[0], ref[0], rtol=1e-12) and np.allclose(got[1], ref[1], rtol=1e-12)
    # the rows of slots left out are not looked at
    away = ~((a["ids"] >= 0) & (a["ids"] < a["E"])).reshape(-1)
    assert away.any()
    a["y"][away] = np.nan
    again = lo.norm_out(**a)
    assert np.array_equal(again[0], got[0]) and np.array_equal(again[1], got[1])


def test_norm_out_reduces_to_the_combine():
    a = _norm_out_args()
    ids, w, y = a["ids"], a["weights"], a["y"]
    out, nxt = lo.norm_out(y, w, ids, a["E"])
    ref = np.einsum("tj,tjh->th", w * ((ids >= 0) & (ids < a["E"])), y.reshape(4, 3, 8))
    assert np.allclose(out, ref) and nxt is None
    assert np.array_equal(lo.norm_out(y)[0], y)          # k = 1, weight 1
    assert np.allclose(lo.norm_out(y, shared=y, gate=np.full(12, -1e4))[0], y)  # gate shut


@pytest.mark.parametrize("mistake", ["k_major", "gate_raw", "scale_residual", "next_of_v"])
def test_norm_out_pins_see_mistakes(mistake):
    a = _norm_out_args()
    ref = _norm_out_loops(a)
    b = dict(a)
    if mistake == "k_major":          # slot j*T + t instead of t*k + j
        b["y"] = a["y"].reshape(4, 3, 8).transpose(1, 0, 2).reshape(12, 8)
    elif mistake == "gate_raw":       # no sigmoid
        b["gate"] = np.log(np.abs(a["gate"]) / np.abs(1 - np.abs(a["gate"])) + 1e-9)
    elif mistake == "scale_residual":
        b["residual"] = a["scale"] * a["residual"]
    else:                             # the next norm without the residual
        b["residual"] = None
    assert not np.allclose(lo.norm_out(**b)[1], ref[1], rtol=1e-3)


def test_router_brute_force():
    r = _rng(3)
    x, w, bias = r.standard_normal((3, 8)), r.standard_normal((5, 8)), r.standard_normal(5)
    got = lo.router_logits(x, w, bias)
    for t in range(3):
        for e in range(5):
            assert math.isclose(got[t, e], sum(x[t, c] * w[e, c] for c in range(8)) + bias[e],
                                rel_tol=1e-12)


def test_lora_brute_force():
    r = _rng(4)
    S, n, K, N, rank = 6, 3, 8, 16, 4
    y, x = r.standard_normal((S, N)), r.standard_normal((S, K))
    a, b, scale = (r.standard_normal((n, rank, K)), r.standard_normal((n, N, rank)),
                   r.standard_normal(n))
    ids = np.array([2, -1, 0, 2, 3, 1])       # -1 and n: no adapter
    got = lo.lora_add(y, x, a, b, ids, scale)
    for s in range(S):
        g = ids[s]
        for c in range(N):
            d = 0.0
            if 0 <= g < n:
                d = scale[g] * sum(b[g, c, q] * sum(a[g, q, h] * x[s, h] for h in range(K))
                                   for q in range(rank))
            assert math.isclose(got[s, c], y[s, c] + d, rel_tol=1e-11, abs_tol=1e-11)
    # the merged weight: y = W x becomes (W + scale B A) x
    W = r.standard_normal((N, K))
    one = lo.lora_add(x @ W.T, x, a[:1], b[:1], np.zeros(S, int), scale[:1])
    assert np.allclose(one, x @ (W + scale[0] * b[0] @ a[0]).T)
