"""Helpers of the tests of the operators around the FFN: inputs, and error bounds
of fp32 arithmetic with one rounding at the end, evaluated with the fp64 values.

u = 2^-24 is fp32's half step relative to a value. A sum of m fp32 terms in any
order is off by at most m u sum|terms| (first order); a product or a sum of two
by u; sqrt and division by u each."""
import numpy as np
import torch

from tests.gpu_util import moe  # noqa: F401

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}   # half a step, relative
TINY = 1e-37                                    # underflow to the subnormal range
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


def rand(g, *shape, dtype="f32", std=1.0):
    return (torch.randn(shape, generator=g) * std).to(DT[dtype]).cuda()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def close(got, ref, err, dtype, what):
    """|got - ref| <= half a step of the output type plus the fp32 error `err`
    (and the half step of that)."""
    got = f64(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.all(np.isfinite(got) == np.isfinite(ref)), what
    tol = HALF[dtype] * np.abs(ref) + 1.01 * err + TINY
    bad = np.abs(got - ref) > tol
    worst = float(np.max(np.abs(got - ref) / tol)) if got.size else 0.0
    print(f"    {what}: largest error {worst:.3f} of its bound", flush=True)
    assert not bad.any(), (what, int(bad.sum()), worst)


def norm_error(v, e_v, weight, eps):
    """fp32 error of rms_norm(v) * weight where v itself is off by e_v: a sum of H
    squares (a thread sums at most 32 of its own, then 6 + 16 steps over lanes and
    waves: 64 covers it), mean, eps, sqrt, reciprocal, two products."""
    ss = np.sum(v * v, 1, keepdims=True)
    inv = 1.0 / np.sqrt(ss / v.shape[1] + eps) if eps else 1.0 / np.sqrt(
        np.maximum(ss, 1e-300) / v.shape[1])
    rel = np.sum(np.abs(v) * e_v, 1, keepdims=True) / np.maximum(ss, 1e-300) + 40 * U
    return (e_v + np.abs(v) * rel) * inv * np.abs(weight)


def sentinel(shape, dtype, pad=64):
    """A tensor inside a larger buffer of sentinel values, and a check that the
    values around it are still there."""
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * pad,), 12345.0, dtype=DT[dtype], device="cuda")

    def intact():
        assert bool((buf[:pad] == 12345.0).all() and (buf[pad + n:] == 12345.0).all()), \
            "written outside the output"
    return buf[pad:pad + n].view(shape), intact
