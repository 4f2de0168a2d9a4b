"""GPU parity of layer norm and its gradients against the fp64 oracle: every output within half a
step of its type plus the fp32 arithmetic's own error."""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo
from tests.gpu_util import moe, say
from tests.layer_util import U, close, f64, gen, rand, sentinel

pytestmark = pytest.mark.gpu
EPS = 1e-5
# a sum over a row: a thread adds up to 32 of its own, then 6 + 16 steps over lanes and waves
ROW = 64 * U

# both sides of every row length's rule, in 16-byte vectors and element by element
SHAPES = [(1, 8, "bf16"), (3, 512, "bf16"), (2, 520, "bf16"), (9, 1024, "bf16"), (4, 1032, "bf16"),
          (3, 2048, "bf16"), (2, 4096, "bf16"), (2, 4104, "bf16"), (3, 7168, "bf16"),
          (2, 8200, "bf16"), (1, 16384, "bf16"), (1, 1, "bf16"), (5, 63, "bf16"), (6, 129, "bf16"),
          (3, 257, "bf16"), (2, 1031, "bf16"), (2, 2049, "bf16"), (1, 4097, "bf16"),
          (1, 16383, "bf16"), (7, 256, "f32"), (2, 1028, "f32"), (2, 4100, "f32"), (2, 8192, "f32"),
          (1, 8196, "f32"), (2, 16384, "f32"), (3, 777, "f32"), (1, 3, "f32"), (2, 16381, "f32"),
          (300, 64, "bf16"), (65, 4096, "bf16"), (515, 200, "f32"), (1030, 72, "bf16"),
          (777, 1031, "f32"), (2100, 136, "bf16"), (40, 12288, "bf16"), (270, 9001, "bf16"),
          (33, 9001, "f32"), (600, 1500, "bf16"), (1100, 2500, "bf16"), (70, 3000, "bf16"),
          (40, 3500, "bf16"), (50, 750, "f32"), (45, 1249, "f32"), (30, 1533, "f32"), (20, 1790, "f32")]


def forward_error(s, e_s, w, b, eps):
    """fp32 error of layer_norm where s itself is off by e_s."""
    H = s.shape[1]
    mean = s.mean(1, keepdims=True)
    e_mean = ROW * np.abs(s).mean(1, keepdims=True) + e_s.mean(1, keepdims=True)
    d = s - mean
    e_d = e_s + e_mean + U * (np.abs(d) + e_s + e_mean)
    var = (d * d).mean(1, keepdims=True) + eps
    e_var = (2 * np.abs(d) * e_d + e_d * e_d).mean(1, keepdims=True) + ROW * var
    inv = 1 / np.sqrt(var)
    # the root's slope is bounded by that at the smallest var the error allows
    low = np.maximum(var - e_var, var * 0.25)
    e_inv = 0.5 * e_var * inv * (var / low) ** 1.5 / var + 4 * U * inv
    u = d * inv
    e_u = e_d * inv + np.abs(d) * e_inv + 2 * U * np.abs(u)
    o = u * np.abs(w)
    return e_u * np.abs(w) + 3 * U * (np.abs(o) + np.abs(b)), (d, e_d, inv, e_inv, u, e_u)


def run_forward(x, res, w, b, alpha, eps, dtype):
    T, H = x.shape
    out, ok = sentinel((T, H), dtype)
    s, ok2 = sentinel((T, H), dtype)
    moe().layer_norm(x, w, b, res, alpha, eps, out=out, residual_out=s)
    torch.cuda.synchronize()
    ok()
    ok2()
    hw = np.ones(H) if w is None else f64(w)
    hb = np.zeros(H) if b is None else f64(b)
    a = np.float32(alpha)
    ref, ref_s = lo.layer_norm(f64(x), hw, hb, None if res is None else f64(res), a, eps)
    e_s = 2 * U * (np.abs(a * f64(x)) + (0 if res is None else np.abs(f64(res))))
    close(s, ref_s, e_s, dtype, "residual_out")
    close(out, ref, forward_error(ref_s, e_s, hw, hb, eps)[0], dtype, "out")
    return out, s


@pytest.mark.parametrize("T,H,dtype", SHAPES)
def test_forward(T, H, dtype):
    say(f"layer_norm T={T} H={H} {dtype}")
    g = gen(T * 7 + H)
    # rows about a mean of their own, as a residual stream's are
    x, res = rand(g, T, H, dtype=dtype), rand(g, T, H, dtype=dtype, std=3.0)
    res += torch.randn((T, 1), generator=g).cuda().to(res.dtype)
    w, b = rand(g, H), rand(g, H)
    out, s = run_forward(x, res, w, b, 0.75, EPS, dtype)
    run_forward(x, None, w, None, -1.25, EPS, dtype)
    run_forward(x, None, None, b, 1.0, 1e-2, dtype)
    run_forward(x, res, None, None, 1.0, EPS, dtype)
    a, c = moe().layer_norm(x, w, b, res, 0.75, EPS)         # the outputs it allocates itself
    assert torch.equal(a, out) and torch.equal(c, s)
    d, none = moe().layer_norm(x, w, b)
    assert none is None and torch.equal(d, moe().layer_norm(x, w, b, eps=1e-5)[0])


def check_backward(dout, s, w, dsum, alpha, eps, got, dtype):
    T, H = s.shape
    hd, hs = f64(dout), f64(s)
    hw = np.ones(H) if w is None else f64(w)
    hr = np.zeros((T, H)) if dsum is None else f64(dsum)
    a = np.float32(alpha)
    dx, ds, dweight, dbias = lo.layer_norm_backward(hd, hs, hw, hr, a, eps)
    _, (d, e_d, inv, e_inv, u, e_u) = forward_error(hs, np.zeros_like(hs), np.ones(H), np.zeros(H),
                                                    eps)
    g = hd * hw
    mg, mgd = g.mean(1, keepdims=True), (g * d).mean(1, keepdims=True)
    e_mg = (ROW + 2 * U) * np.abs(g).mean(1, keepdims=True)
    e_mgd = (np.abs(g) * e_d).mean(1, keepdims=True) + (ROW + 3 * U) * np.abs(g * d).mean(
        1, keepdims=True)
    mgu = mgd * inv
    e_mgu = e_mgd * inv + np.abs(mgd) * e_inv + 2 * U * np.abs(mgu)
    inner = np.abs(g) + np.abs(mg) + np.abs(u * mgu)
    e_inner = 5 * U * inner + e_mg + e_u * np.abs(mgu) + np.abs(u) * e_mgu
    e_ds = e_inner * inv + inner * e_inv + 3 * U * (inner * inv + np.abs(hr))
    close(got[0], dx, np.abs(a) * e_ds + 2 * U * np.abs(dx), dtype, "dx")
    if got[1] is not None:
        close(got[1], ds, e_ds, dtype, "dresidual")
    if got[2] is not None:
        close(got[2], dweight, (T + 4) * U * np.abs(hd * u).sum(0) + (np.abs(hd) * e_u).sum(0),
              "f32", "dweight")
    if got[3] is not None:
        close(got[3], dbias, (T + 2) * U * np.abs(hd).sum(0), "f32", "dbias")


@pytest.mark.parametrize("T,H,dtype", SHAPES)
def test_backward(T, H, dtype):
    say(f"layer_norm_backward T={T} H={H} {dtype}")
    g = gen(T * 5 + H)
    s = rand(g, T, H, dtype=dtype, std=2.0) + torch.randn((T, 1), generator=g).cuda().to(
        rand(g, 1, dtype=dtype).dtype)
    dout, dsum, w = (rand(g, T, H, dtype=dtype), rand(g, T, H, dtype=dtype), rand(g, H))
    bufs = [sentinel((T, H), dtype), sentinel((T, H), dtype), sentinel((H,), "f32"),
            sentinel((H,), "f32")]
    dx, dr, dw, db = (b[0] for b in bufs)
    # a workspace of whatever values
    n = moe().layer_norm_backward_workspace_bytes(T, H)
    ws = torch.full((n + 64,), 0x7f, dtype=torch.uint8, device="cuda")
    got = moe().layer_norm_backward(dout, s, w, dsum, 0.75, EPS, dx, dr, dw, db, ws)
    torch.cuda.synchronize()
    for _, ok in bufs:
        ok()
    assert bool((ws[n:] == 0x7f).all()), "written past the workspace"
    check_backward(dout, s, w, dsum, 0.75, EPS, got, dtype)
    own = moe().layer_norm_backward(dout, s, w, dsum, 0.75, EPS)
    assert all(torch.equal(a, b) for a, b in zip(got, own))
    # without a weight and a residual
    got = moe().layer_norm_backward(dout, s, eps=1e-2)
    assert got[1] is None and got[2] is None
    check_backward(dout, s, None, None, 1.0, 1e-2, got, dtype)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 40, 257])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sums_over_rows(T, dtype):
    """One workgroup or several, rows of one wave or of more, and gradients of weight and bias off
    the 16-byte grid, each with and without the other."""
    say(f"layer_norm_backward: sums T={T} {dtype}")
    m = moe()
    for H in (5, 9, 64, 257, 509, 512, 1000, 1023, 1032, 2056, 4099, 9000):
        g = gen(T + H)
        s, dout, w = rand(g, T, H, dtype=dtype, std=2.0), rand(g, T, H, dtype=dtype), rand(g, H)
        ref = m.layer_norm_backward(dout, s, w, eps=EPS)
        check_backward(dout, s, w, None, 1.0, EPS, ref, dtype)
        off = torch.full((2, H + 2), 12345.0, device="cuda")
        m.layer_norm_backward(dout, s, w, eps=EPS, dweight=off[0, 1:H + 1], dbias=off[1, 1:H + 1])
        assert torch.equal(off[0, 1:H + 1], ref[2]) and torch.equal(off[1, 1:H + 1], ref[3])
        assert bool((off[:, [0, H + 1]] == 12345.0).all())
        ws = torch.empty(m.layer_norm_backward_workspace_bytes(T, H), dtype=torch.uint8,
                         device="cuda")
        for only in (0, 1):
            one = torch.full((H,), 12345.0, device="cuda")
            dx = torch.empty_like(dout)
            to = [one.data_ptr() if i == only else None for i in (0, 1)]
            status = m.lib.moe_layer_norm_backward(
                dout.data_ptr(), s.data_ptr(), w.data_ptr(), None, 1.0, EPS, T, H,
                {"bf16": 1, "f32": 0}[dtype], dx.data_ptr(), None, *to, ws.data_ptr(), ws.numel(),
                torch.cuda.current_stream().cuda_stream)
            assert status == 0 and torch.equal(one, ref[2 + only]) and torch.equal(dx, ref[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(dtype):
    say(f"layer_norm in place {dtype}")
    g, m = gen(1), moe()
    for H in (1032, 1031):
        x, res = rand(g, 9, H, dtype=dtype), rand(g, 9, H, dtype=dtype)
        w, b, dout = rand(g, H), rand(g, H), rand(g, 9, H, dtype=dtype)
        out, s = m.layer_norm(x, w, b, res, 0.5, EPS)
        x1, r1 = x.clone(), res.clone()
        m.layer_norm(x1, w, b, r1, 0.5, EPS, out=x1, residual_out=r1)
        assert torch.equal(x1, out) and torch.equal(r1, s)
        x2, r2 = x.clone(), res.clone()
        m.layer_norm(x2, w, b, r2, 0.5, EPS, out=r2, residual_out=x2)
        assert torch.equal(r2, out) and torch.equal(x2, s)
        ref = m.layer_norm_backward(dout, s, w, res, 0.5, EPS)
        for dx, dr in ((0, 1), (1, 2), (2, 0)):
            t = [dout.clone(), s.clone(), res.clone()]
            got = m.layer_norm_backward(t[0], t[1], w, t[2], 0.5, EPS, dx=t[dx], dresidual=t[dr])
            assert all(torch.equal(a, c) for a, c in zip(got, ref)), (H, dx, dr)


def test_special_rows():
    say("layer_norm: rows of one value, infinities, NaN stay in their rows")
    m, H = moe(), 264
    x = torch.randn(6, H, generator=gen(2)).bfloat16().cuda()
    x[1] = 3
    x[3, 7] = float("inf")
    x[4, 100] = float("nan")
    w, b = torch.ones(H, device="cuda"), torch.full((H,), 0.25, device="cuda")
    out, _ = m.layer_norm(x, w, b, eps=EPS)
    zero, _ = m.layer_norm(x, w, b, eps=0.0)
    assert bool((out[1] == 0.25).all()) and bool(torch.isnan(zero[1]).all())
    assert bool(torch.isnan(out[3:5]).all()) and bool(torch.isfinite(out[[0, 1, 2, 5]]).all())
    ref, _ = m.layer_norm(x[[0, 2, 5]].contiguous(), w, b, eps=EPS)
    assert torch.equal(out[[0, 2, 5]], ref)
    dout = torch.randn(6, H, generator=gen(3)).bfloat16().cuda()
    dx, _, dw, db = m.layer_norm_backward(dout, x, w, eps=EPS)
    assert bool(torch.isnan(dx[3:5]).all()) and bool(torch.isfinite(dx[[0, 1, 2, 5]]).all())
    assert bool(torch.isnan(dw).all()) and bool(torch.isfinite(db).all())


def test_no_rows():
    say("layer_norm: no rows")
    m = moe()
    e = torch.empty((0, 72), device="cuda")
    w = torch.ones(72, device="cuda")
    out, s = m.layer_norm(e, w, w, residual=e)
    assert out.shape == s.shape == (0, 72)
    dw, db = torch.full((72,), 5.0, device="cuda"), torch.full((72,), 5.0, device="cuda")
    m.layer_norm_backward(e, e, w, dweight=dw, dbias=db)
    torch.cuda.synchronize()
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_rows_far_from_zero():
    """A mean of 1000 beside a spread of 1: squares about the mean, not of the values."""
    say("layer_norm: a large mean")
    g = gen(4)
    x = (torch.randn(5, 1000, generator=g) + 1000).cuda()
    w, b = rand(g, 1000), rand(g, 1000)
    run_forward(x, None, w, b, 1.0, EPS, "f32")
    dout = rand(g, 5, 1000)
    got = moe().layer_norm_backward(dout, x, w, eps=EPS)
    check_backward(dout, x, w, None, 1.0, EPS, got, "f32")


def test_gradient_against_differences():
    """The derivative along a direction, from the GPU's own forward calls in fp32: with a step h the
    difference quotient is off by the third derivative's share, O(h^2), which falls by four when h
    is halved and is taken out by (4 q(h/2) - q(h)) / 3; what is left is O(h^4) and the rounding of
    the outputs over h."""
    say("layer_norm gradients against differences")
    m, g = moe(), gen(5)
    T, H, eps = 4, 512, 0.1
    x, v, dout = rand(g, T, H), rand(g, T, H), rand(g, T, H)
    w = rand(g, H)

    def loss(t, wt):
        return float((m.layer_norm(t, wt, eps=eps)[0].double() * dout.double()).sum())

    def slope(f):
        q = [(f(h) - f(-h)) / (2 * h) for h in (0.125, 0.0625)]
        return (4 * q[1] - q[0]) / 3

    dx, _, dw, _ = m.layer_norm_backward(dout, x, w, eps=eps)
    got = float((dx.double() * v.double()).sum())
    num = slope(lambda h: loss(x + h * v, w))
    # rounding: T H outputs of size one, u each and at random, over h; O(h^4): outputs change by
    # their own size over a step of one, so h^4 of the sum of the terms' sizes
    size = float((dx.double() * v.double()).abs().sum())
    tol = 64 * U * np.sqrt(T * H) * float(dout.abs().max()) / 0.0625 + 0.125 ** 4 * size
    say(f"    {got:.6f} against {num:.6f}, bound {tol:.2e}")
    assert abs(got - num) <= tol
    # the weight enters linearly: no truncation, the rounding of x + h v is not there either
    q = rand(g, H)
    got = float((dw.double() * q.double()).sum())
    num = slope(lambda h: loss(x, w + h * q))
    size = float((dw.double() * q.double()).abs().sum())
    assert abs(got - num) <= 64 * U * np.sqrt(T * H) * float(dout.abs().max()) / 0.0625 + 1e-4 * size


def test_offsets_past_32_bits():
    T, H = (1 << 18) + 5, 16384
    say(f"layer_norm {T} x {H} bf16")
    m = moe()
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x[-3:] = rand(gen(6), 3, H, dtype="bf16")
    last = x[-3:].clone()
    w = rand(gen(7), H)
    out, _ = m.layer_norm(x, w, eps=EPS)
    ref, _ = m.layer_norm(last, w, eps=EPS)
    assert torch.equal(out[-3:], ref)
    dx, _, dw, db = m.layer_norm_backward(out, x, w, eps=EPS, dx=out)
    one = m.layer_norm_backward(ref, last, w, eps=EPS)
    assert torch.equal(dx[-3:], one[0])
    # all other rows add zeros
    assert torch.allclose(db, one[3], rtol=1e-5, atol=1e-5)
