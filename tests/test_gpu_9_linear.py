"""GPU parity of the matrix product with its epilogue against the fp64 oracle: every output within
half a step of its type plus the fp32 arithmetic's own error."""
import math

import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo
from tests.gpu_util import moe, say
from tests.layer_util import DT, U, close, f64, gen, rand, sentinel

pytestmark = pytest.mark.gpu
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def act_code(name):
    m = moe()
    return {"none": m.ACT_NONE, "relu": m.ACT_RELU, "silu": m.ACT_SILU, "gelu": m.ACT_GELU,
            "gelu_tanh": m.ACT_GELU_TANH}[name]


def act_error(act, v, e):
    """Error of the activation of v that is off by e: no slope exceeds 1.2; exp, erf and the steps
    after them are off by less than 8 u of v (a gelu far below zero is the small difference of
    terms as large as v)."""
    return e if act in ("none", "relu") else 1.2 * e + 8 * U * np.abs(v)


def check(x, w, bias, act, gated, res, out, dtype, what="out"):
    hx, hw = f64(x), f64(w)
    hb = None if bias is None else f64(bias)
    hr = None if res is None else f64(res)
    K, n = hx.shape[1], hw.shape[0]
    v = hx @ hw.T
    e = (K + 2) * U * (np.abs(hx) @ np.abs(hw).T)
    if hb is not None:
        v = v + hb
        e += U * np.abs(hb)
    if gated:
        N = n // 2
        a, u = lo.activate(act, v[:, :N]), v[:, N:]
        ea = act_error(act, v[:, :N], e[:, :N])
        e = ea * np.abs(u) + np.abs(a) * e[:, N:] + ea * e[:, N:] + U * np.abs(a * u)
    else:
        e = act_error(act, v, e)
    ref = lo.linear(hx, hw, hb, act, gated, hr)
    close(out, ref, e + 2 * U * np.abs(ref), dtype, what)


def run(T, N, K, act="none", gated=False, bias=False, res=False, dtype="bf16", odt=None, seed=None):
    odt = odt or dtype
    say(f"linear T={T} N={N} K={K} {act} gated={gated} bias={bias} res={res} {dtype} -> {odt}")
    g = gen(T * 3 + N * 7 + K if seed is None else seed)
    n = 2 * N if gated else N
    x, w = rand(g, T, K, dtype=dtype), rand(g, n, K, dtype=dtype, std=K ** -0.5)
    b = rand(g, n) if bias else None
    r = rand(g, T, N, dtype=odt, std=2.0) if res else None
    out, ok = sentinel((T, N), odt)
    need = moe().linear_workspace_bytes(T, N, K, gated, {"bf16": 1, "f32": 0}[dtype])
    ws = torch.full((need + 256,), 0x7f, dtype=torch.uint8, device="cuda")
    moe().linear(x, w, b, act_code(act), gated, r, out=out, workspace=ws)
    torch.cuda.synchronize()
    ok()
    assert bool((ws[need:] == 0x7f).all()), "written past the workspace"
    check(x, w, b, act, gated, r, out, odt)
    own = moe().linear(x, w, b, act_code(act), gated, r, dtype=DT[odt])
    assert torch.equal(own, out)
    return x, w, b, r, out


# tokens on both sides of every rule, odd widths, K with a partial chunk of 64 at its end
SIZES = [(1, 1, 8), (1, 64, 64), (1, 4096, 72), (2, 17, 200), (3, 4, 1000), (7, 129, 264),
         (8, 128, 512), (9, 96, 4096), (16, 2048, 1032), (17, 33, 136), (24, 1000, 8),
         (31, 256, 2048), (32, 65, 64), (33, 64, 128), (48, 520, 328), (63, 127, 1024),
         (64, 1536, 520), (65, 300, 96), (100, 100, 104), (127, 511, 256), (128, 64, 4104),
         (129, 1, 40), (200, 2050, 192), (255, 256, 64), (256, 257, 320), (300, 384, 1000),
         (400, 96, 2048), (511, 130, 72), (513, 640, 136), (640, 1100, 64), (777, 333, 264),
         (1024, 512, 200), (1025, 1025, 128), (2047, 65, 88), (2500, 260, 56)]


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sizes(T, N, K, dtype):
    # what is on changes from case to case, so that all meet across them
    q = T + N
    run(T, N, K, ACTS[q % 5], q % 3 == 0, q % 2 == 0, q % 4 < 2, dtype,
        ("bf16", "f32", dtype)[q % 3])


@pytest.mark.parametrize("K", [8, 16, 24, 32, 40, 56])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_shorter_than_a_stage(K, dtype):
    """Several rows lie within the bytes that a stage takes of one, also behind the last."""
    for T, N, gated in ((130, 70, False), (300, 131, True), (65, 33, True), (513, 257, False)):
        run(T, N, K, "relu", gated, True, True, dtype)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,N,K", [(5, 76, 200), (40, 131, 264), (300, 260, 136), (700, 516, 72)])
def test_epilogues(act, gated, T, N, K):
    for bias in (False, True):
        for res in (False, True):
            run(T, N, K, act, gated, bias, res, "bf16", "bf16" if bias else "f32")
    run(T, N, K, act, gated, True, True, "f32")


@pytest.mark.parametrize("T", [1, 4, 16, 40, 64, 128, 400, 1000, 2304])
@pytest.mark.parametrize("N,K,gated", [(2048, 1024, True), (4096, 512, False), (1288, 4096, False)])
def test_wide(T, N, K, gated):
    run(T, N, K, "silu", gated, True, not gated)


@pytest.mark.parametrize("T", [3, 50, 300, 700])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_in_place(T, dtype):
    """x, residual and out as column slices of wider matrices (out and residual off the vectors'
    alignment too), out over residual; nothing beside the columns is written."""
    say(f"linear slices T={T} {dtype}")
    m, g = moe(), gen(T)
    N, K = 90, 136
    wide = rand(g, T, K + 24, dtype=dtype)
    x = wide[:, 16:16 + K]
    w, b = rand(g, N, K, dtype=dtype, std=K ** -0.5), rand(g, N)
    rwide = rand(g, T, 3 * N + 2, dtype=dtype)
    for at in (0, 4, 5):
        res = rwide[:, at:at + N]
        big = torch.full((T, 2 * N + 7), 12345.0, dtype=DT[dtype], device="cuda")
        out = big[:, at:at + N]
        m.linear(x, w, b, m.ACT_SILU, residual=res, out=out)
        check(x.contiguous(), w, b, "silu", False, res, out, dtype)
        keep = torch.ones(2 * N + 7, dtype=torch.bool)
        keep[at:at + N] = False
        assert bool((big[:, keep.cuda()] == 12345.0).all())
        again = rwide.clone()
        over = again[:, at:at + N]
        m.linear(x, w, b, m.ACT_SILU, residual=over, out=over)
        assert torch.equal(over, out)
        keep = torch.ones(3 * N + 2, dtype=torch.bool)
        keep[at:at + N] = False
        assert torch.equal(again[:, keep.cuda()], rwide[:, keep.cuda()])
    # out beside x in one matrix
    both = torch.zeros((T, K + N + 6), dtype=DT[dtype], device="cuda")
    both[:, :K] = x
    if (K + N + 6) % 8 == 0:
        m.linear(both[:, :K], w, out=both[:, K:K + N])
        assert torch.equal(both[:, K:K + N], m.linear(x, w))


@pytest.mark.parametrize("T,N,K", [(3, 70, 264), (40, 200, 1032), (300, 150, 264), (700, 300, 72)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_special_values_stay_in_their_rows(T, N, K, dtype):
    say(f"linear: infinities and NaN T={T} N={N} K={K} {dtype}")
    m, g = moe(), gen(8)
    x, w = rand(g, T, K, dtype=dtype), rand(g, N, K, dtype=dtype)
    clean = m.linear(x, w)
    x1, w1 = x.clone(), w.clone()
    x1[1, 3], x1[T - 1, K - 1] = float("nan"), float("inf")
    w1[5, 0], w1[N - 1, K - 2] = float("inf"), float("nan")
    out = m.linear(x1, w1)
    rows = torch.ones(T, dtype=torch.bool)
    rows[[1, T - 1]] = False
    cols = torch.ones(N, dtype=torch.bool)
    cols[[5, N - 1]] = False
    fine = rows.cuda()[:, None] & cols.cuda()[None]
    assert bool((~torch.isfinite(out[~fine])).all())
    assert torch.equal(out[fine], clean[fine])
    b = torch.zeros(N, device="cuda")
    b[7] = float("nan")
    for act in (m.ACT_NONE, m.ACT_RELU, m.ACT_SILU, m.ACT_GELU, m.ACT_GELU_TANH):
        out = m.linear(x, w, b, act)
        assert bool(torch.isnan(out[:, 7]).all()) and bool(torch.isfinite(out[:, :7]).all())
        assert bool(torch.isfinite(out[:, 8:]).all())


def test_activations_far_out():
    """Products of any size: exp and its like leave the fp32 range without a NaN."""
    say("linear: activations of large values")
    m = moe()
    v = torch.tensor([-3e38, -1e30, -1e4, -100.0, -90.0, -20.0, -0.0, 0.0, 20.0, 100.0, 1e4, 1e30,
                      3e38], device="cuda")
    x = torch.zeros((1, 8), device="cuda")
    x[0, 0] = 1
    w = torch.zeros((13, 8), device="cuda")
    w[:, 0] = v
    assert torch.equal(m.linear(x, w)[0], v)
    relu = m.linear(x, w, activation=m.ACT_RELU)[0]
    assert torch.equal(relu, v.clamp(min=0))
    for act in (m.ACT_SILU, m.ACT_GELU, m.ACT_GELU_TANH):
        out = m.linear(x, w, activation=act)[0]
        assert bool(torch.isfinite(out).all()) and torch.equal(out[8:], v[8:]), out
        assert bool((out[:6].abs() <= 1e-6).all()), out


@pytest.mark.parametrize("T", [6, 40, 300, 700])
def test_fp32_loses_no_bits(T):
    """Whole numbers of 24 bits times one and zero: exact, whatever the kernel does with fp32. Less
    their first 16 bits they are exact too as long as the sum on the way stays in 24 bits: taken
    away in pieces of 8 bits, the second of which is at most 2^15 (half a step of the first for
    values below 2^24), it does where |x| <= 2^24 - 2^15; past that it may pass 2^24, where fp32
    counts in twos, and be off by 1."""
    say(f"linear: 24-bit values T={T}")
    m, g = moe(), gen(9)
    K, N = 264, 264
    x = torch.randint(-(1 << 24) + 1, 1 << 24, (T, K), generator=g).float().cuda()
    pick = torch.randperm(K, generator=g)
    w = torch.zeros((N, K), device="cuda")
    w[torch.arange(N), pick] = 1
    assert torch.equal(m.linear(x, w), x[:, pick.cuda()])
    # the sum of such a value and its first 16 bits taken away
    top = (x.view(torch.int32) & ~0xff).view(torch.float32)
    x2 = torch.cat([x, top], 1)
    w2 = torch.cat([w, -w], 1)
    off = (m.linear(x2, w2) - (x - top)[:, pick.cuda()]).abs()
    edge = x[:, pick.cuda()].abs() > (1 << 24) - (1 << 15)
    assert bool((off[~edge] == 0).all()) and bool((off[edge] <= 1).all())


@pytest.mark.parametrize("T,N,K", [(5, 200, 4096), (60, 300, 8192), (500, 256, 4096),
                                   (1500, 512, 2048)])
def test_fp32_rms(T, N, K):
    """Random fp32 operands, in units of u times the sum's size, sqrt(K) products of size one. One
    chain of K additions rounds sums of size sqrt(i), i = 1 .. K, each by a uniform error within
    half a step: a step is 2 u times the power of two below the sum, so the error's rms is
    2 u / sqrt(12) of that power, 0.40 u of a sum spread over its octave (the mean of 1 / m^2 over
    m in [1, 2) with density 1 / (m ln 2) is 0.54, its root 0.74, less 2 / sqrt(12) = 0.58 of it:
    0.43). The squares add up to 0.43^2 u^2 K^2 / 2: 0.30 sqrt(K) u, 19.5 at K = 4096. Shorter chains
    make less. A fifth on top for the sample; a lost plane of eight bits would be 40 and more."""
    say(f"linear: fp32 rms T={T} N={N} K={K}")
    g = gen(10)
    x, w = rand(g, T, K), rand(g, N, K)
    err = f64(moe().linear(x, w)) - f64(x) @ f64(w).T
    rms = float(np.sqrt((err * err).mean()) / (U * np.sqrt(K)))
    say(f"    rms {rms:.2f} u")
    assert rms <= 1.2 * 0.30 * np.sqrt(K)


def test_rows_do_not_meet():
    """A row's bits do not depend on the other rows' values, for equal sizes."""
    say("linear: rows on their own")
    m, g = moe(), gen(11)
    for T in (16, 60, 300, 700):
        x, w = rand(g, T, 264, dtype="bf16"), rand(g, 300, 264, dtype="bf16")
        a = m.linear(x, w)
        x2 = rand(g, T, 264, dtype="bf16")
        x2[T // 2] = x[T // 2]
        assert torch.equal(m.linear(x2, w)[T // 2], a[T // 2])


def test_no_tokens():
    m = moe()
    w = torch.ones((9, 64), device="cuda")
    assert m.linear(torch.empty((0, 64), device="cuda"), w).shape == (0, 9)


def test_offsets_past_32_bits():
    """Weights of more than 2^32 bytes, and rows of x and out past 2^31 elements; the last rows and
    columns are checked."""
    m, g = moe(), gen(12)
    N, K = 600007, 4096
    say(f"linear: w {N} x {K} bf16")
    w = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
    w[-40:] = rand(g, 40, K, dtype="bf16", std=K ** -0.5)
    for T in (3, 70):
        x = rand(g, T, K, dtype="bf16")
        out = m.linear(x, w)
        check(x, w[-40:], None, "none", False, None, out[:, -40:], "bf16")
        assert bool((out[:, :-40] == 0).all())
    x = rand(g, 5, K, dtype="bf16")
    even = w[:-1]
    out = m.linear(x, even, activation=m.ACT_RELU, gated=True)   # gate and up rows 2.4 GB apart
    half = even.shape[0] // 2
    pair = torch.cat([even[half - 40:half], even[-40:]])
    check(x, pair, None, "relu", True, None, out[:, -40:], "bf16")
    del w, even, out
    T = 600011
    say(f"linear: x {T} x {K}, out {T} x 4096")
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    x[-70:] = rand(g, 70, K, dtype="bf16")
    w = rand(g, 4096, K, dtype="bf16", std=K ** -0.5)
    out = m.linear(x, w)
    check(x[-70:], w, None, "none", False, None, out[-70:], "bf16")
    assert bool((out[:-70] == 0).all())


# fp32 tiles of all three sizes (the last two: 1024 x 4096 and 2048 x 4096 w rows are 256 of them)
@pytest.mark.parametrize("T,N", [(300, 520), (1024, 4096), (2048, 4096)])
@pytest.mark.parametrize("gated", [False, True])
def test_fp32_of_one_sign(T, N, gated):
    """Positive operands and eight products a sum: nothing averages out, and fp32 has nearly all
    bits of the sum. Of a product 2^-23 = 2 u may be left out; the first planes' products have 16
    bits, so that eight of them between 1 and 4 add up exactly, and go with the rest (all other
    pairs of planes, below 2^-6 of them, whose own steps count for 0.1 u) into one step of the
    sum, 2 u whichever way it is rounded: 4.1 u of the sum. Planes cut off after 8 bits each leave
    7.8 u out for operands of 1 + 2^-7 - 2^-23. The few-rows kernel takes the same planes in the
    same order: the two differ by no more than 0.1 u in the mean (planes cut off: 0.6)."""
    say(f"linear: fp32 of one sign T={T} N={N} gated={gated}")
    m, g, K = moe(), gen(13), 8
    n = N // 2 if gated else N

    def run_(x, w):
        if not gated:
            return m.linear(x, w)
        b = torch.cat([torch.zeros(n), torch.ones(n)]).cuda()     # gate times one
        return m.linear(x, torch.cat([w[:n], torch.zeros_like(w[:n])]), b, gated=True)

    worst = torch.full((1, K), 1 + 2.0 ** -7 - 2.0 ** -23, device="cuda")
    some = [1 + torch.rand((r, K), generator=g).cuda() for r in (T, N)]
    for x, w in ((worst.repeat(T, 1), worst.repeat(N, 1)), some):
        ref = f64(x) @ f64(w[:n]).T
        off = np.abs(f64(run_(x, w)) - ref).max() / U / ref.min()
        say(f"    {off:.2f} u")
        assert np.all(np.abs(f64(run_(x, w)) - ref) <= 4.1 * U * ref)
    x, w = some
    d = f64(run_(x, w)[:16]) - f64(run_(x[:16].contiguous(), w))
    mean = float((d / (f64(x[:16]) @ f64(w[:n]).T)).mean()) / U
    say(f"    mean difference from the few-rows kernel {mean:.3f} u")
    assert abs(mean) <= 0.1


@pytest.mark.parametrize("T,N", [(300, 520), (1024, 4096), (2048, 4096)])
def test_fp32_ends_of_the_range(T, N):
    """The largest fp32 values (which round to a bf16 infinity) stay what they are in tiles, and of
    the smallest what is not below 2^-133."""
    say(f"linear: ends of the fp32 range T={T} N={N}")
    m, g, K = moe(), gen(14), 264
    pick = torch.randint(0, K, (N,), generator=g)
    w = torch.zeros((N, K), device="cuda")
    w[torch.arange(N), pick] = 0.5
    last = torch.randint(0x7f7f0000, 0x7f800000, (T, K), generator=g).int().cuda().view(torch.float32)
    last[0, :2] = torch.tensor([3.4028234663852886e38, -3.4028234663852886e38])
    last[1::2] *= -1
    # (one such value a row: the others' products with 0 are zeros)
    assert torch.equal(m.linear(last, w), last[:, pick.cuda()] * 0.5)
    small = torch.randint(-(1 << 24) + 1, 1 << 24, (T, K), generator=g).float().cuda() * 2.0 ** -133
    assert torch.equal(m.linear(small, 2 * w), small[:, pick.cuda()])


@pytest.mark.parametrize("T", [1, 100])
def test_gelu_of_one_value(T):
    """GELU of exact products in fp32, also where it is the small difference of large terms. Its
    tail, erfc(|v| / sqrt 2) / 2, is off by (20 + v^2) u of itself at most: the reciprocal and its
    operand 3 u, which count 2.3 times; 1 - t 1 u; the polynomial's steps 7 u and fit 0.4; the
    exponential 2 u, its argument v^2 u; two products 2 u. Below zero the result is v times that
    (1 u more), above v times one less it (2 u)."""
    say(f"linear: gelu T={T}")
    m, g = moe(), gen(15)
    v = torch.cat([12.5 * (2 * torch.rand(3000, generator=g) - 1),
                   2 * torch.rand(3000, generator=g) - 1,
                   10.0 ** (-30 * torch.rand(500, generator=g)),
                   -10.0 ** (-30 * torch.rand(500, generator=g))]).cuda()
    x, w = torch.zeros((T, 8), device="cuda"), torch.zeros((v.numel(), 8), device="cuda")
    x[:, 0], w[:, 0] = 1, v
    assert torch.equal(m.linear(x, w)[T // 2], v)
    out, h = f64(m.linear(x, w, activation=m.ACT_GELU)), f64(v)
    tail = 0.5 * np.vectorize(math.erfc)(np.abs(h) / math.sqrt(2))
    ref = np.where(h < 0, h * tail, h * (1 - tail))
    tol = np.abs(h) * (tail * (20 + h * h) + np.where(h < 0, tail, 2)) * U
    worst = float((np.abs(out - ref) / tol).max())
    say(f"    largest error {worst:.3f} of its bound")
    assert worst <= 1


# few rows of every size; every tile, whole K and K in parts; K past a chunk and a stage by 8 or more
EXACT = [(1, 4100, 4104), (7, 300, 8), (9, 2048, 1000), (16, 2050, 7176), (29, 1001, 2056),
         (64, 512, 520), (64, 2048, 7176), (70, 70, 8184), (300, 520, 4104), (700, 700, 8200),
         (512, 4096, 1032), (1024, 4096, 1000), (3000, 1500, 2008), (2048, 4096, 1096),
         (4096, 4099, 328)]


@pytest.mark.parametrize("T,N,K", EXACT)
@pytest.mark.parametrize("gated", [False, True])
def test_bf16_whole_numbers(T, N, K, gated):
    """Whole numbers to 8 in bf16: every sum stays below 64 K < 2^24 and is exact in fp32 in any
    order, so that one k too few or too many shows. Gated: gate or up sums of K products, the
    other one's of a single one, 2^22 at most together."""
    say(f"linear: whole numbers T={T} N={N} K={K} gated={gated}")
    m, g = moe(), torch.Generator("cuda").manual_seed(T + N + K)

    def whole(rows):
        return torch.randint(-8, 9, (rows, K), generator=g, device="cuda").bfloat16()

    x, w = whole(T), whole(N)
    ref = x.double() @ w.double().T
    if not gated:
        assert torch.equal(m.linear(x, w, dtype=torch.float32).double(), ref)
        return
    pick = torch.randint(0, K, (N,), generator=g, device="cuda")
    one = torch.zeros_like(w)
    one[torch.arange(N, device="cuda"), pick] = 1
    ref *= x[:, pick].double()
    assert float(ref.abs().max()) < 2 ** 24
    for pair in ((w, one), (one, w)):
        got = m.linear(x, torch.cat(pair), gated=True, dtype=torch.float32)
        assert torch.equal(got.double(), ref)
