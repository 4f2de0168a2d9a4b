"""GPU parity of the adapters of many requests against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo
from tests.gpu_util import moe, say
from tests.layer_util import DT, U, close, f64, gen, rand

pytestmark = pytest.mark.gpu


def _inputs(S, n, r, K, N, xdt="bf16", ydt="bf16", seed=0, ids=None):
    g = gen(seed + S + 31 * n + r + K + N)
    if ids is None:
        ids = torch.randint(-1, n, (S,), generator=g)
    return dict(ids=ids.int().cuda().view(S, 1), x=rand(g, S, K, dtype=xdt),
                a=rand(g, n, r, K, dtype="bf16", std=K ** -0.5),
                b=rand(g, n, N, r, dtype="bf16"), scale=rand(g, n),
                y=rand(g, S, N, dtype=ydt))


def _run(d, block_m, out=None, scale=True, **kw):
    plan = moe().align_block(d["ids"], d["a"].shape[0], block_m)
    return moe().lora_add(d["y"] if out is None else d["y"], d["x"], d["a"], d["b"], *plan,
                          block_m, scale=d["scale"] if scale else None, out=out, **kw)


def _check(d, got, y, scale=True):
    ids = d["ids"].view(-1).cpu().numpy()
    n, r, K = d["a"].shape
    x, a, b = f64(d["x"]), f64(d["a"]), f64(d["b"])
    sc = f64(d["scale"]) if scale else None
    ref = lo.lora_add(f64(y), x, a, b, ids, sc)
    # z: a sum of K products in fp32 (of fp32 x: kept to 2^-23); the expansion: a sum of r
    # products, of z to 16 bits for a bf16 output and to 23 for fp32; scale; the last sum
    zero = np.zeros_like(ref)
    mag = lo.lora_add(zero, np.abs(x), np.abs(a), np.abs(b), ids,
                      None if sc is None else np.abs(sc))
    dt = "bf16" if d["y"].dtype == torch.bfloat16 else "f32"
    e = (K + r + 8) * U * mag + (2.0 ** -16 * mag if dt == "bf16" else 0) + U * np.abs(f64(y))
    close(got, ref, e, dt, "out")
    away = (ids < 0) | (ids >= n)
    assert torch.equal(got[torch.from_numpy(away).cuda()], y[torch.from_numpy(away).cuda()])


CASES = [  # S, n, r, K, N, block_m
    (1, 1, 8, 8, 8, 1), (1, 1, 16, 4096, 4096, 64), (2, 3, 8, 64, 136, 16), (7, 5, 24, 72, 72, 4),
    (16, 16, 16, 4096, 1024, 64), (16, 4, 64, 520, 2056, 16), (33, 2, 40, 1032, 264, 2),
    (64, 64, 128, 256, 512, 64), (64, 1, 256, 264, 520, 64), (65, 3, 32, 2048, 64, 128),
    (130, 7, 16, 136, 4104, 256), (300, 1, 64, 512, 512, 256), (300, 200, 8, 128, 256, 64),
    (511, 1024, 16, 256, 264, 64), (1000, 9, 96, 1000, 1000, 64), (520, 8, 128, 64, 2048, 8),
    (200, 3, 248, 200, 200, 32),
    # few rows of an adapter with ranks above 32; many slices of K
    (7, 5, 64, 72, 520, 16), (6, 4, 256, 136, 264, 64), (9, 9, 40, 1032, 200, 2),
    (3, 2, 16, 8264, 72, 64), (5, 3, 128, 4096, 136, 64), (2, 1, 64, 8192, 72, 16),
    # b shared between rows or not: 2 and 8 rows an adapter, 16 and 17 adapters, rank 64 on
    (32, 16, 16, 136, 264, 64), (31, 16, 16, 136, 264, 64), (136, 17, 8, 72, 264, 64),
    (135, 17, 8, 72, 264, 64), (40, 17, 64, 72, 264, 64), (8, 4, 72, 72, 264, 64),
    # one launch or two: 512 readings of a
    (600, 512, 8, 72, 264, 64), (600, 513, 8, 72, 264, 64), (300, 171, 24, 72, 200, 64),
    (300, 170, 24, 72, 200, 64), (200, 128, 32, 136, 1024, 64), (200, 129, 32, 136, 1024, 64),
    (20, 20, 32, 136, 1032, 64), (256, 256, 16, 200, 2056, 16), (3, 3, 24, 4168, 1032, 1),
    # thirty-two rows an adapter or fewer
    (12, 3, 32, 136, 264, 64), (11, 3, 32, 136, 264, 64), (96, 3, 8, 520, 136, 64),
    (95, 3, 8, 520, 136, 64), (160, 40, 24, 72, 72, 32),
    # thirty-two rows at a time in the shrink
    (4100, 2, 64, 520, 264, 64), (4100, 3, 16, 200, 136, 32), (4095, 2, 24, 136, 72, 256),
    (4200, 1, 160, 136, 328, 64),
    # few workgroups of the shrink: 16 ranks each, groups of 16 rows below 8 groups of 64
    (28, 1, 128, 936, 360, 64), (80, 6, 64, 1520, 1000, 64), (90, 11, 40, 1032, 136, 64),
    (30, 3, 24, 200, 136, 256)]


@pytest.mark.parametrize("S,n,r,K,N,block_m", CASES)
@pytest.mark.parametrize("xdt,ydt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"),
                                     ("f32", "bf16")])
def test_lora_parity(S, n, r, K, N, block_m, xdt, ydt):
    say(f"lora S={S} n={n} r={r} K={K} N={N} M={block_m} {xdt}->{ydt}")
    d = _inputs(S, n, r, K, N, xdt, ydt)
    y = d["y"].clone()
    out = torch.empty_like(y).copy_(y)
    assert _run(d, block_m, out=out) is out
    torch.cuda.synchronize()
    assert torch.equal(d["y"], y), "y is an input here"
    _check(d, out, y)
    got = _run(d, block_m)                                # in place
    assert got is d["y"] and torch.equal(got, out)        # the same bits
    d["y"] = y.clone()
    _check(d, _run(d, block_m, scale=False), y, scale=False)


@pytest.mark.parametrize("kind", ["none", "one_row", "all_one", "last", "out_of_range"])
def test_lora_uneven_batches(kind):
    say(f"lora ids: {kind}")
    S, n = 150, 6
    ids = torch.full((S,), -1)
    if kind == "one_row":
        ids[77] = 3
    elif kind == "all_one":
        ids[:] = 2
    elif kind == "last":
        ids[-3:] = n - 1
    elif kind == "out_of_range":
        ids[:] = torch.arange(S) % 9 - 2                   # -2..6: some beyond n - 1
    d = _inputs(S, n, 16, 264, 392, ids=ids)
    away = (ids < 0) | (ids >= n)
    d["x"][away.cuda()] = float("nan")                     # rows without an adapter are not read
    d["y"][away.cuda()] = 7.0
    y = d["y"].clone()
    got = _run(d, 16)
    d["x"][away.cuda()] = 0
    _check(d, got, y)


@pytest.mark.parametrize("r", [8, 16, 24, 32, 40])
@pytest.mark.parametrize("S,n", [(100, 20), (620, 600)])
def test_lora_one_popular_adapter(S, n, r):
    # many rows of one adapter where the sizes let few be expected
    say(f"lora: S={S} n={n} r={r}, one adapter for almost all")
    ids = torch.full((S,), 7)
    ids[5::17] = n - 1
    ids[3::29] = -1
    d = _inputs(S, n, r, 136, 328, ids=ids)
    y = d["y"].clone()
    _check(d, _run(d, 64, out=d["y"].clone()), y)
    _check(d, _run(d, 8), y)


@pytest.mark.parametrize("M", [16, 32, 64, 256])
@pytest.mark.parametrize("S,n,r", [(500, 100, 8), (500, 100, 16), (500, 400, 32), (500, 100, 64),
                                   (60, 8, 24), (55, 7, 72), (33, 5, 128), (14, 9, 16)])
def test_lora_runs_of_rows(S, n, r, M):
    # a few adapters with whole blocks of rows each, beside many with one or none: less
    # than eight groups, more, and numbers that eight does not divide
    say(f"lora: runs of rows, S={S} n={n} r={r} M={M}")
    g = gen(S + n)
    ids = torch.randint(0, n, (6,), generator=g)[torch.arange(S) * 6 // S]
    ids[::7] = torch.randint(-1, n, (len(ids[::7]),), generator=g)
    d = _inputs(S, n, r, 200, 136, ids=ids)
    y = d["y"].clone()
    _check(d, _run(d, M, out=d["y"].clone()), y)


@pytest.mark.parametrize("xdt,ydt", [("bf16", "bf16"), ("f32", "f32")])
def test_lora_column_slices(xdt, ydt):
    # x, y and out as column slices of wider matrices; what lies beside them stays
    say(f"lora: strided rows {xdt} {ydt}")
    S, n, r, K, N = 70, 4, 16, 264, 200
    d = _inputs(S, n, r, K, N, xdt, ydt)
    ref = torch.empty_like(d["y"]).copy_(d["y"])
    _run(d, 16, out=ref)
    wide_x = torch.full((S, K + 24), float("nan"), dtype=DT[xdt], device="cuda")
    wide_y = torch.full((S, 3 * N), 5.0, dtype=DT[ydt], device="cuda")
    wide_x[:, 16:16 + K] = d["x"]
    wide_y[:, N:2 * N] = d["y"]
    s = {**d, "x": wide_x[:, 16:16 + K], "y": wide_y[:, N:2 * N]}
    out = torch.full((S, N + 40), 6.0, dtype=DT[ydt], device="cuda")
    view = out[:, 8:8 + N]
    view.copy_(d["y"])
    _run(s, 16, out=view)
    assert torch.equal(view, ref) and bool((out[:, :8] == 6).all() and (out[:, 8 + N:] == 6).all())
    _run(s, 16)
    assert torch.equal(wide_y[:, N:2 * N], ref)
    assert bool((wide_y[:, :N] == 5).all() and (wide_y[:, 2 * N:] == 5).all())


def test_lora_non_finite_stay_in_their_rows():
    say("lora: infinities and NaN")
    d = _inputs(40, 3, 24, 200, 136)
    d["ids"] = (torch.arange(40) % 3).int().cuda().view(40, 1)
    y = d["y"].clone()
    ref = _run(d, 16, out=torch.empty_like(y)).clone()
    x = d["x"].clone()
    d["x"][5, 7] = float("nan")
    d["x"][9, 100] = float("inf")
    got = _run(d, 16, out=torch.empty_like(y)).clone()
    keep = torch.ones(40, dtype=torch.bool)
    keep[[5, 9]] = False
    assert torch.equal(got[keep.cuda()], ref[keep.cuda()])
    assert not bool(torch.isfinite(got[[5, 9]]).any())
    d["x"] = x
    d["a"][1, 3, 20] = float("inf")                        # an adapter that overflowed
    got = _run(d, 16, out=torch.empty_like(y))
    assert torch.equal(got[0::3], ref[0::3]) and torch.equal(got[2::3], ref[2::3])
    assert not bool(torch.isfinite(got[1::3]).any())


@pytest.mark.parametrize("r", [8, 16, 24, 64])
def test_lora_non_finite_factor_columns(r):
    # an infinity in b belongs to its own output column of its adapter's rows
    say(f"lora: an infinity in b, r={r}")
    d = _inputs(20, 2, r, 72, 264, ids=torch.arange(20) % 2)
    y = d["y"].clone()
    ref = _run(d, 16, out=torch.empty_like(y)).clone()
    d["b"][1, 77, 3] = float("inf")
    got = _run(d, 16, out=torch.empty_like(y))
    assert not bool(torch.isfinite(got[1::2, 77]).any())
    got[1::2, 77] = ref[1::2, 77]
    assert torch.equal(got, ref)


def test_lora_workspace_of_a_larger_batch():
    # one workspace for the largest batch serves every smaller one; nothing is
    # read that the call did not write
    say("lora: one workspace")
    n, r, K, N = 3, 40, 1032, 136
    sizes = [300, 1, 17, 64, 2, 299]
    need = max(moe().lora_workspace_bytes(S, n, K, r, 64) for S in sizes)
    assert need == moe().lora_workspace_bytes(300, n, K, r, 64)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN in fp32
    for S in sizes:
        d = _inputs(S, n, r, K, N)
        y = d["y"].clone()
        ws.fill_(0xFF)
        _check(d, _run(d, 64, workspace=ws), y)


@pytest.mark.parametrize("S,r", [(70, 40), (70, 16), (12, 40), (12, 16), (600, 16)])
def test_lora_lists_in_another_order(S, r):
    # empty places before a block's rows: the same rows, and nothing out of place
    say(f"lora: lists whose blocks do not hold their rows first, S={S} r={r}")
    n = 257 if S == 600 else 3
    d = _inputs(S, n, r, 72, 136)
    M = 16
    ids, blocks, padded = moe().align_block(d["ids"], n, M)
    ids = ids[:ids.numel() // M * M].view(-1, M).flip(1).reshape(-1).contiguous()
    need = moe().lora_workspace_bytes(S, n, 72, r, M)
    buf = torch.full((need + 65536,), 77, dtype=torch.uint8, device="cuda")
    y = d["y"].clone()
    ref = _run({**d, "y": y.clone()}, M)
    moe().lora_add(d["y"], d["x"], d["a"], d["b"], ids, blocks, padded, M, scale=d["scale"],
                   workspace=buf[:need])
    torch.cuda.synchronize()
    assert bool((buf[need:] == 77).all())
    assert torch.equal(d["y"], ref)
    away = (d["ids"].view(-1) < 0)
    assert torch.equal(d["y"][away], y[away])


def test_lora_empty_and_checks():
    say("lora: S=0, binding checks")
    m = moe()
    d = _inputs(20, 3, 16, 64, 128)
    plan = m.align_block(d["ids"], 3, 16)
    e = m.lora_add(d["y"][:0], d["x"][:0], d["a"], d["b"], *plan, 16)
    assert e.shape == (0, 128)
    call = lambda **kw: m.lora_add(**{**dict(  # noqa: E731
        y=d["y"], x=d["x"], a=d["a"], b=d["b"], sorted_ids=plan[0], block_adapter=plan[1],
        num_padded=plan[2], block_m=16, scale=d["scale"]), **kw})
    y = d["y"].clone()
    for kw in (dict(y=d["y"][:19]), dict(x=d["x"][:, :56]), dict(b=d["b"][:2]),
               dict(b=d["b"][:, :120].contiguous()), dict(scale=d["scale"][:2]),
               dict(x=d["x"].t()), dict(out=y[:, :64]), dict(block_m=64),
               dict(sorted_ids=plan[0][:8]), dict(y=d["y"].cpu()), dict(x=d["x"][:, ::2]),
               dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
               dict(y=d["y"][0].expand(20, 128))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(a=d["a"].float()), dict(b=d["b"].half()), dict(scale=d["scale"].bfloat16()),
               dict(out=y.float()), dict(y=d["y"].half())):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(m.MoEError):
        call(x=torch.zeros((20, 72), dtype=torch.bfloat16, device="cuda")[:, 4:68])  # 8 bytes off
    torch.cuda.synchronize()
    assert torch.equal(d["y"], y)


def test_lora_more_groups_than_a_grid_row():
    say("lora: 70000 rows in blocks of one")
    d = _inputs(70000, 3, 8, 8, 16)
    y = d["y"].clone()
    _check(d, _run(d, 1), y)


def test_lora_refuses_out_over_x():
    say("lora: out over x, adapters on a matrix itself")
    m = moe()
    d = _inputs(20, 3, 16, 64, 64)
    plan = m.align_block(d["ids"], 3, 16)
    x = d["x"].clone()
    with pytest.raises(m.MoEError):
        m.lora_add(d["x"], d["x"], d["a"], d["b"], *plan, 16)
    torch.cuda.synchronize()
    assert torch.equal(d["x"], x)
    out = m.lora_add(d["x"], d["x"], d["a"], d["b"], *plan, 16, out=x.clone())   # y = x
    _check({**d, "y": x, "scale": d["scale"]}, out, x, scale=False)


def test_lora_rows_past_32_bit_offsets():
    # slices of a matrix of more than 2^31 elements
    S, n, K, N, wide = 40000, 2, 64, 64, 65536
    say(f"lora S={S} in rows of {wide}")
    d = _inputs(S, n, 8, K, N)
    d["ids"][1:-5] = -1
    d["ids"][-5:] = 1
    big = torch.zeros((S, wide), dtype=torch.bfloat16, device="cuda")
    assert big.numel() > 2 ** 31
    big[:, wide - N:] = d["y"]
    y = d["y"].clone()
    d["y"] = big[:, wide - N:]
    got = _run(d, 64)
    torch.cuda.synchronize()
    _check({**d, "y": y}, got.contiguous(), y)
    assert not bool(big[-8:, :wide - N].any())
