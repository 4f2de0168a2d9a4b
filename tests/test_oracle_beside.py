"""Pins of the fp64 oracle of the operators beside the FFN: brute-force loops on tiny
shapes, closed forms, and the gradients against differences of the forward functions."""
import math

import numpy as np
import pytest

import oracle
from oracle import layer_oracle as lo


def _rng(seed):
    return np.random.default_rng(seed)


def _routing(seed, T=5, k=3, E=6, local=4, M=4):
    r = _rng(seed)
    ids = np.stack([r.permutation(E)[:k] for _ in range(T)])
    sid, _, n = oracle.align(ids, local, M)
    return ids, sid, n, lo.places(sid, n, T * k).reshape(T, k)


def differences(f, x, h=1e-5):
    """Gradient of the scalar f at x by central differences."""
    x = np.array(x, np.float64)
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_places_and_dispatch_by_hand():
    # two experts, runs padded to 2; slot 1 is another shard's
    sid = np.array([0, 3, 2, 4, 4, 4])
    assert lo.places(sid, 4, 4).tolist() == [0, -1, 2, 1]
    rows = lo.dispatch(np.array([[1.0, 2.0], [3.0, 4.0]]), sid, 4, 2)
    assert rows.tolist() == [[1, 2], [3, 4], [3, 4], [0, 0]]


def test_dispatch_holds_each_token_at_its_experts_run():
    ids, sid, n, at = _routing(0)
    x = _rng(1).standard_normal((5, 7))
    rows = lo.dispatch(x, sid, n, 3)
    seen = set()
    for t in range(5):
        for j in range(3):
            assert (at[t, j] < 0) == (ids[t, j] >= 4)
            if at[t, j] >= 0:
                assert np.array_equal(rows[at[t, j]], x[t])
                seen.add(at[t, j])
    for p in range(n):
        assert p in seen or not rows[p].any()


def test_combine_loops_and_closed_form():
    ids, sid, n, at = _routing(2)
    r = _rng(3)
    rows, w = r.standard_normal((n, 4)), r.random((5, 3))
    out = lo.combine(rows, at, w)
    for t in range(5):
        for c in range(4):
            v = math.fsum(w[t, j] * rows[at[t, j], c] for j in range(3) if at[t, j] >= 0)
            assert math.isclose(out[t, c], v, rel_tol=1e-13, abs_tol=1e-15)
    # a token's copies summed give it once for each of its places
    x = r.standard_normal((5, 4))
    assert np.allclose(lo.combine(lo.dispatch(x, sid, n, 3), at),
                       x * (at >= 0).sum(1)[:, None])


def test_gradients_of_dispatch_and_combine_against_differences():
    ids, sid, n, at = _routing(4)
    r = _rng(5)
    x, w = r.standard_normal((5, 3)), r.random((5, 3))
    seed_rows, dout = r.standard_normal((n, 3)), r.standard_normal((5, 3))
    dx = differences(lambda v: np.sum(seed_rows * lo.dispatch(v, sid, n, 3)), x)
    assert np.allclose(lo.combine(seed_rows, at), dx, atol=1e-8)
    rows = r.standard_normal((n, 3))
    drows, dw = lo.combine_backward(dout, rows, at, w, n)
    assert np.allclose(drows, differences(lambda v: np.sum(dout * lo.combine(v, at, w)), rows),
                       atol=1e-8)
    assert np.allclose(dw, differences(lambda v: np.sum(dout * lo.combine(rows, at, v)), w),
                       atol=1e-8)


def test_layer_norm_closed_forms():
    out, s = lo.layer_norm(np.array([[1.0, 3.0], [5.0, 5.0]]), np.array([2.0, 3.0]),
                           np.array([10.0, 20.0]), eps=0.25)
    q = 1 / math.sqrt(1.25)
    assert np.allclose(out, [[10 - 2 * q, 20 + 3 * q], [10, 20]]) and s[0, 1] == 3.0
    # a constant added to a row, or without eps a positive factor, changes nothing
    x = _rng(6).standard_normal((2, 9))
    a, _ = lo.layer_norm(x, eps=0.0)
    assert np.allclose(lo.layer_norm(3 * x + 7, eps=0.0)[0], a)
    assert np.allclose(a.mean(1), 0) and np.allclose((a * a).mean(1), 1)


def test_layer_norm_brute_force():
    r = _rng(7)
    x, res, w, b = (r.standard_normal(sh) for sh in ((3, 5), (3, 5), 5, 5))
    out, s = lo.layer_norm(x, w, b, res, alpha=-0.5, eps=1e-3)
    for t in range(3):
        row = [res[t, c] - 0.5 * x[t, c] for c in range(5)]
        m = math.fsum(row) / 5
        q = math.sqrt(math.fsum((v - m) ** 2 for v in row) / 5 + 1e-3)
        for c in range(5):
            assert math.isclose(s[t, c], row[c], rel_tol=1e-13)
            assert math.isclose(out[t, c], (row[c] - m) / q * w[c] + b[c], rel_tol=1e-11,
                                abs_tol=1e-13)


@pytest.mark.parametrize("affine", [True, False])
def test_layer_norm_gradients_against_differences(affine):
    r = _rng(8)
    x, res, w, b = (r.standard_normal(sh) for sh in ((3, 6), (3, 6), 6, 6))
    dout, dsum = r.standard_normal((3, 6)), r.standard_normal((3, 6))
    weight, bias = (w, b) if affine else (None, None)

    def loss(xv, rv, wv, bv):
        out, s = lo.layer_norm(xv, wv, bv, rv, alpha=0.75, eps=1e-2)
        return np.sum(out * dout) + np.sum(s * dsum)

    _, s = lo.layer_norm(x, weight, bias, res, alpha=0.75, eps=1e-2)
    dx, ds, dw, db = lo.layer_norm_backward(dout, s, weight, dsum, alpha=0.75, eps=1e-2)
    assert np.allclose(dx, differences(lambda v: loss(v, res, weight, bias), x), atol=1e-7)
    assert np.allclose(ds, differences(lambda v: loss(x, v, weight, bias), res), atol=1e-7)
    one, zero = (w, b) if affine else (np.ones(6), np.zeros(6))
    assert np.allclose(dw, differences(lambda v: loss(x, res, v, zero), one), atol=1e-7)
    assert np.allclose(db, differences(lambda v: loss(x, res, one, v), zero), atol=1e-7)


def test_activations():
    v = np.array([-30.0, -1.0, 0.0, 1.0, 30.0])
    assert lo.activate("relu", v).tolist() == [0, 0, 0, 1, 30]
    sig = 1 / (1 + math.exp(-1.0))
    assert np.allclose(lo.activate("silu", v), [-30 * math.exp(-30), sig - 1, 0, sig, 30])
    phi = 0.5 * (1 + math.erf(math.sqrt(0.5)))          # the normal distribution at 1
    assert np.allclose(lo.activate("gelu", v), [0, phi - 1, 0, phi, 30])
    t = 0.5 * (1 + math.tanh(math.sqrt(2 / math.pi) * 1.044715))
    assert np.allclose(lo.activate("gelu_tanh", v), [0, t - 1, 0, t, 30])
    # the two gelus are one function to within 5e-4
    x = np.linspace(-6, 6, 400)
    assert 1e-5 < np.abs(lo.activate("gelu", x) - lo.activate("gelu_tanh", x)).max() < 5e-4


@pytest.mark.parametrize("gated", [False, True])
def test_linear_loops(gated):
    r = _rng(9)
    n = 6 if gated else 3
    x, w, b, res = (r.standard_normal(sh) for sh in ((2, 5), (n, 5), n, (2, 3)))
    out = lo.linear(x, w, b, "silu", gated, res)
    for t in range(2):
        for c in range(3):
            g = math.fsum(x[t, i] * w[c, i] for i in range(5)) + b[c]
            v = g / (1 + math.exp(-g))
            if gated:
                v *= math.fsum(x[t, i] * w[3 + c, i] for i in range(5)) + b[3 + c]
            assert math.isclose(out[t, c], res[t, c] + v, rel_tol=1e-12)


def test_planted_mistakes_are_seen():
    """Each pin above tells the definition from a near miss of it."""
    r = _rng(10)
    x, w = r.standard_normal((3, 6)), r.standard_normal(6)
    out, _ = lo.layer_norm(x, w, eps=1e-2)
    d = x - x.mean(1, keepdims=True)
    unbiased = d / np.sqrt((d * d).sum(1, keepdims=True) / 5 + 1e-2) * w
    no_mean = x / np.sqrt((x * x).mean(1, keepdims=True) + 1e-2) * w
    assert not np.allclose(out, unbiased) and not np.allclose(out, no_mean)
    g = r.standard_normal((3, 6))
    _, ds, dw, _ = lo.layer_norm_backward(g, x, w, eps=1e-2)
    inv = 1 / np.sqrt((d * d).mean(1, keepdims=True) + 1e-2)
    gw = g * w
    assert not np.allclose(ds, inv * (gw - gw.mean(1, keepdims=True)))
    assert not np.allclose(ds, inv * (g - g.mean(1, keepdims=True)
                                      - d * inv * (g * d * inv).mean(1, keepdims=True)))
    assert not np.allclose(dw, (gw * d * inv).sum(0))
