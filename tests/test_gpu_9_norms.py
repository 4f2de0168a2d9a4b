"""GPU parity of the norms around the block against the fp64 oracle: every
output within half a step of its type plus the fp32 arithmetic's own error."""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo
from tests.gpu_util import moe, say
from tests.layer_util import U, close, f64, gen, norm_error, rand, sentinel

pytestmark = pytest.mark.gpu
EPS = 1e-5

# rows of one wave (four to a workgroup), of four and of sixteen, on and off their limits
SHAPES = [(1, 8, "bf16"), (3, 16, "bf16"), (5, 136, "bf16"), (9, 512, "bf16"), (2, 520, "bf16"),
          (6, 1024, "bf16"), (4, 1032, "bf16"), (3, 2048, "bf16"), (2, 4096, "bf16"),
          (2, 4104, "bf16"), (3, 7168, "bf16"), (1, 8200, "bf16"), (2, 16384, "bf16"),
          (7, 256, "f32"), (1, 4, "f32"), (5, 12, "f32"), (3, 1028, "f32"), (2, 2052, "f32"),
          (2, 4100, "f32"), (2, 8188, "f32"), (1, 16380, "f32"), (2, 16384, "f32"),
          (300, 64, "bf16"), (65, 4096, "bf16"),
          # two vectors per thread from 512 rows on
          (511, 4360, "bf16"), (512, 4360, "bf16"), (513, 2300, "f32")]


def _check_in(x, res, w, alpha, out, s_out, dtype, eps=EPS):
    ref, s = lo.norm_in(f64(x), f64(w), None if res is None else f64(res), np.float32(alpha), eps)
    # fp32 product and sum: within 2 u of the sum of the magnitudes
    mag = np.abs(np.float32(alpha) * f64(x)) + (0 if res is None else np.abs(f64(res)))
    e_s = 2 * U * mag
    close(out, ref, norm_error(s, e_s, f64(w), eps), dtype, "out")
    if s_out is not None:
        close(s_out, s, e_s, dtype, "residual_out")


@pytest.mark.parametrize("T,H,dtype", SHAPES)
def test_norm_in_parity(T, H, dtype):
    say(f"norm_in T={T} H={H} {dtype}")
    g = gen(T * 7 + H)
    x, res = rand(g, T, H, dtype=dtype), rand(g, T, H, dtype=dtype, std=3.0)
    w = rand(g, H)
    for r, alpha in ((res, 0.5), (res, -1.25), (None, 1.0)):
        out, ok1 = sentinel((T, H), dtype)
        s, ok2 = sentinel((T, H), dtype)
        moe().norm_in(x, w, r, alpha, EPS, out=out, residual_out=s)
        torch.cuda.synchronize()
        ok1()
        ok2()
        _check_in(x, r, w, alpha, out, s, dtype)
    a, b = moe().norm_in(x, w, res, -1.25, EPS)      # the outputs it allocates itself
    c, none = moe().norm_in(x, w)
    assert none is None
    _check_in(x, res, w, -1.25, a, b, dtype)
    _check_in(x, None, w, 1.0, c, None, dtype, eps=1e-6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_in_in_place(dtype):
    say(f"norm_in in place {dtype}")
    g = gen(1)
    x, res, w = rand(g, 9, 1032, dtype=dtype), rand(g, 9, 1032, dtype=dtype), rand(g, 1032)
    out, s = moe().norm_in(x, w, res, 0.5, EPS)
    x1, r1 = x.clone(), res.clone()
    moe().norm_in(x1, w, r1, 0.5, EPS, out=x1, residual_out=r1)
    assert torch.equal(x1, out) and torch.equal(r1, s)
    x2, r2 = x.clone(), res.clone()
    moe().norm_in(x2, w, r2, 0.5, EPS, out=r2, residual_out=x2)
    assert torch.equal(r2, out) and torch.equal(x2, s)


def test_norm_special_rows():
    say("norm: zero rows, infinities, NaN stay in their rows")
    x = torch.randn(6, 264, generator=gen(2)).bfloat16().cuda()
    x[1] = 0
    x[3, 7] = float("inf")
    x[4, 100] = float("nan")
    w = torch.ones(264, device="cuda")
    out, _ = moe().norm_in(x, w, eps=EPS)
    z, _ = moe().norm_in(x, w, eps=0.0)
    o, n = moe().norm_out(x, next_weight=w, weight=w, eps=EPS)
    torch.cuda.synchronize()
    assert bool((out[1] == 0).all()) and bool(torch.isnan(z[1]).all())
    assert bool((o[1] == 0).all()) and bool((n[1] == 0).all())
    for t in (out, o, n):
        assert bool(torch.isnan(t[4]).all()) and bool(torch.isnan(t[3, 7]))
        assert bool(torch.isfinite(t[[0, 1, 2, 5]]).all())
    ref, _ = moe().norm_in(x[[0, 2, 5]].contiguous(), w, eps=EPS)
    assert torch.equal(out[[0, 2, 5]], ref)


def _args_out(T, k, H, ydt, dt, seed, E=8, local=None, shared=True, gate=True, residual=True,
              weight=True, nxt=True, ids=True, weights=True):
    g = gen(seed)
    local = E if local is None else local
    a = dict(y=rand(g, T * k, H, dtype=ydt))
    # any ids at all, also repeated and negative ones
    a["topk_ids"] = torch.randint(-2, E, (T, k), generator=g).int().cuda() if ids else None
    a["num_experts"] = local if ids else None
    a["topk_weights"] = torch.rand((T, k), generator=g).cuda() if weights else None
    a["shared"] = rand(g, T, H, dtype=dt) if shared else None
    a["gate"] = rand(g, T, std=2.0) if gate else None
    a["residual"] = rand(g, T, H, dtype=dt, std=3.0) if residual else None
    a["weight"] = rand(g, H) if weight else None
    a["next_weight"] = rand(g, H) if nxt else None
    return a


def _check_out(a, scale, out, nxt, dt, eps=EPS):
    h = {n: None if t is None else (t if isinstance(t, int) else f64(t)) for n, t in a.items()}
    ids = None if a["topk_ids"] is None else a["topk_ids"].cpu().numpy()
    sc = np.float32(scale)
    ref, ref_n = lo.norm_out(h["y"], h["topk_weights"], ids, h["num_experts"], h["shared"],
                             h["gate"], h["residual"], h["weight"], h["next_weight"], sc, eps)
    # errors, step by step: sums of k + 1 products, the sigmoid (exp, sum, division: 4 u)
    away = {n: h[n] for n in ("topk_weights", "shared", "gate")}
    v, _ = lo.norm_out(h["y"], away["topk_weights"], ids, h["num_experts"], away["shared"],
                       away["gate"])
    mag, _ = lo.norm_out(np.abs(h["y"]), away["topk_weights"], ids, h["num_experts"],
                         None if h["shared"] is None else np.abs(h["shared"]), away["gate"])
    k = 1 if h["topk_weights"] is None else h["topk_weights"].shape[1]
    e = (k + 8) * U * mag
    n = v
    if h["weight"] is not None:
        e = norm_error(v, e, h["weight"], eps)
        n = lo.rms_norm(v, h["weight"], eps)
    e = np.abs(sc) * e + 3 * U * (np.abs(sc * n) + (0 if h["residual"] is None
                                                    else np.abs(h["residual"])))
    close(out, ref, e, dt, "out")
    if h["next_weight"] is not None:
        close(nxt, ref_n, norm_error(ref, e, h["next_weight"], eps), dt, "next")


OUT_SHAPES = [(1, 1, 8, "bf16", "bf16"), (5, 2, 136, "bf16", "bf16"), (3, 8, 1024, "bf16", "bf16"),
              (2, 8, 4096, "bf16", "bf16"), (3, 6, 4104, "bf16", "bf16"),
              (2, 8, 7168, "f32", "bf16"), (1, 3, 16384, "f32", "bf16"),
              (4, 2, 520, "bf16", "f32"), (2, 5, 2048, "bf16", "f32"), (3, 2, 12, "f32", "f32"),
              (2, 4, 4100, "f32", "f32"), (2, 2, 16380, "f32", "f32"), (5, 1, 264, "f32", "f32"),
              (2, 65, 264, "bf16", "bf16"), (3, 130, 64, "f32", "bf16"), (130, 8, 512, "bf16", "bf16"),
              (70, 8, 4096, "bf16", "bf16")]


@pytest.mark.parametrize("T,k,H,ydt,dt", OUT_SHAPES)
def test_norm_out_parity(T, k, H, ydt, dt):
    say(f"norm_out T={T} k={k} H={H} y {ydt} {dt}")
    full = dict(T=T, k=k, H=H, ydt=ydt, dt=dt)
    for i, (opts, scale) in enumerate([
            ({}, 0.5), (dict(weight=False), -1.5), (dict(shared=False, gate=False), 1.0),
            (dict(gate=False, nxt=False), 2.0), (dict(residual=False, ids=False), 1.0),
            (dict(shared=False, gate=False, residual=False, weight=False, nxt=False), 1.0)]):
        a = _args_out(**full, seed=T + H + i, **opts)
        out, ok1 = sentinel((T, H), dt)
        nxt, ok2 = sentinel((T, H), dt)
        moe().norm_out(**a, scale=scale, eps=EPS, out=out,
                       next_out=nxt if a["next_weight"] is not None else None)
        torch.cuda.synchronize()
        ok1()
        ok2()
        if a["next_weight"] is None:
            assert bool((nxt == nxt[0, 0]).all())           # not written
        _check_out(a, scale, out, nxt, dt)


def test_norm_out_leaves_other_shards_alone():
    # rows of slots outside [0, E) hold NaN; a token with no slot here keeps its residual
    say("norm_out: slots of other shards")
    a = _args_out(12, 4, 1032, "bf16", "bf16", 5, E=16, local=4, shared=False, gate=False)
    a["topk_ids"][3] = 4
    a["topk_ids"][7] = -1
    a["topk_ids"][8] = torch.tensor([3, 2, 1, 0])
    ids = a["topk_ids"]
    away = (ids < 0) | (ids >= 4)
    clean = {**a, "y": a["y"].clone()}
    clean["y"][away.reshape(-1)] = 0
    a["y"][away.reshape(-1)] = float("nan")
    out, nxt = moe().norm_out(**a, scale=0.5, eps=EPS)
    torch.cuda.synchronize()
    assert torch.equal(out[[3, 7]], a["residual"][[3, 7]])
    assert bool(torch.isfinite(out.float()).all() and torch.isfinite(nxt.float()).all())
    _check_out(clean, 0.5, out, nxt, "bf16")


def test_norm_out_in_place_and_gate_range():
    say("norm_out in place; gates far out")
    a = _args_out(6, 3, 520, "bf16", "bf16", 9)
    a["gate"] = torch.tensor([-200.0, 200.0, 0.0, -float("inf"), float("inf"), -88.0],
                             device="cuda")
    out, nxt = moe().norm_out(**a, scale=0.5, eps=EPS)
    _check_out(a, 0.5, out, nxt, "bf16")
    b = {**a, "residual": a["residual"].clone(), "shared": a["shared"].clone()}
    moe().norm_out(**b, scale=0.5, eps=EPS, out=b["residual"], next_out=b["shared"])
    assert torch.equal(b["residual"], out) and torch.equal(b["shared"], nxt)
    b = {**a, "residual": a["residual"].clone(), "shared": a["shared"].clone()}
    moe().norm_out(**b, scale=0.5, eps=EPS, out=b["shared"], next_out=b["residual"])
    assert torch.equal(b["shared"], out) and torch.equal(b["residual"], nxt)


def test_norm_out_defaults_and_three_dim_y():
    say("norm_out: k = 1 without weights, y as [T, k, H]")
    a = _args_out(6, 1, 264, "bf16", "bf16", 11, shared=False, gate=False, ids=False,
                  weights=False)
    out, nxt = moe().norm_out(**a, eps=EPS)
    _check_out(a, 1.0, out, nxt, "bf16")
    b = _args_out(6, 4, 264, "bf16", "bf16", 12)
    out, nxt = moe().norm_out(**b, eps=EPS)
    out3, nxt3 = moe().norm_out(**{**b, "y": b["y"].view(6, 4, 264)}, eps=EPS)
    assert torch.equal(out, out3) and torch.equal(nxt, nxt3)
    # the combine of moe_ffn_*: equal to its fp32 sum in the order of the slots
    c = _args_out(6, 4, 264, "f32", "f32", 13, shared=False, gate=False, residual=False,
                  weight=False, nxt=False)
    out, none = moe().norm_out(**c)
    assert none is None
    _check_out(c, 1.0, out, None, "f32")


def test_norm_out_infinite_weight_counts_once():
    # rows of 3 slots (fewer than are loaded together), the last one's weight infinite:
    # infinities of y's signs, no NaN from the places of slots that are not there
    say("norm_out: an infinite weight")
    y = rand(gen(14), 3 * 3, 136, dtype="f32")
    w = torch.tensor([[0.5, 0.25, float("inf")], [1.0, 2.0, 3.0], [0.5, 0.25, -float("inf")]],
                     device="cuda")
    out, _ = moe().norm_out(y, w)
    inf = float("inf")
    assert torch.equal(out[0], torch.sign(y[2]) * inf)
    assert torch.equal(out[2], torch.sign(y[8]) * -inf)
    assert bool(torch.isfinite(out[1]).all())


def test_norm_empty_batch():
    say("norms T=0")
    x, w = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), torch.ones(64, device="cuda")
    out, res = moe().norm_in(x, w, x)
    assert out.shape == res.shape == (0, 64)
    out, nxt = moe().norm_out(x, torch.empty((0, 2), device="cuda"), next_weight=w)
    assert out.shape == nxt.shape == (0, 64)


def test_norm_out_rows_past_32_bit_offsets():
    # y holds more than 2^31 elements; the last tokens' rows lie beyond
    T, k, H = 33000, 8, 8192
    say(f"norm_out T={T} k={k} H={H}")
    y = torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda")
    y[-k:] = torch.arange(1, k + 1, device="cuda").view(k, 1).bfloat16()
    y[:k] = 2
    w = torch.full((T, k), 0.5, device="cuda")
    out, _ = moe().norm_out(y, w)
    torch.cuda.synchronize()
    assert y.numel() > 2 ** 31
    assert bool((out[-1] == 18).all()) and bool((out[0] == 8).all()) and not bool(out[1:-1].any())


@pytest.mark.parametrize("T,k,H,ydt,dt", [(2100, 8, 4104, "bf16", "bf16"),
                                          (4200, 8, 1032, "f32", "bf16")])
def test_norm_out_streamed(T, k, H, ydt, dt):
    # y beyond the size up to which it is read through the caches
    say(f"norm_out T={T} k={k} H={H} y {ydt}, streamed")
    a = _args_out(T, k, H, ydt, dt, 21, E=16, local=12)
    assert a["y"].numel() * a["y"].element_size() > 128 << 20
    out, nxt = moe().norm_out(**a, scale=0.5, eps=EPS)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out.float()).all() and torch.isfinite(nxt.float()).all())
    rows = torch.tensor([0, 1, 63, 64, T // 2, T - 2, T - 1])
    pick = {n: t if t is None or isinstance(t, int) or n in ("weight", "next_weight")
            else t.view(T, k * H)[rows.cuda()].view(-1, H) if n == "y" else t[rows.cuda()]
            for n, t in a.items()}
    _check_out(pick, 0.5, out[rows.cuda()], nxt[rows.cuda()], dt)


@pytest.mark.parametrize("T,H", [((1 << 22) + 7, 8), ((1 << 20) + 3, 1032)])
def test_norm_rows_past_the_first_grid_row(T, H):
    say(f"norm_in T={T} H={H}")
    x = torch.full((T, H), 2.0, dtype=torch.bfloat16, device="cuda")
    x[-1] = -3
    w = torch.arange(1, H + 1, device="cuda").float()
    out, _ = moe().norm_in(x, w, eps=0.0)
    torch.cuda.synchronize()
    assert torch.equal(out[-1], (-w).bfloat16())
    assert bool((out[:-1] == w.bfloat16()).all())
    o, _ = moe().norm_out(x, residual=x)
    assert torch.equal(o, 2 * x)


def test_norm_argument_checks():
    say("norms: binding checks")
    m = moe()
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda"), torch.ones(64, device="cuda")
    k2, i2 = torch.ones((4, 2), device="cuda"), torch.zeros((4, 2), dtype=torch.int32,
                                                           device="cuda")
    y2 = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    bad = [lambda: m.norm_in(x, w[:32]), lambda: m.norm_in(x, w, x[:3]),
           lambda: m.norm_in(x[:, ::2], w[:32]), lambda: m.norm_in(x, w, out=x[:2]),
           lambda: m.norm_in(x, w.cpu()), lambda: m.norm_out(y2, k2[:3]),
           lambda: m.norm_out(y2, k2, i2), lambda: m.norm_out(y2, k2, i2[:3], 4),
           lambda: m.norm_out(y2, k2, shared=x[:3]), lambda: m.norm_out(y2, k2, residual=y2),
           lambda: m.norm_out(y2, k2, weight=w[:8])]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: m.norm_in(x, w.bfloat16()), lambda: m.norm_in(x, w, x.float()),
              lambda: m.norm_out(y2, k2, shared=x, residual=x.float()),
              lambda: m.norm_out(y2, k2, dtype=torch.float16),
              lambda: m.norm_out(y2, k2.bfloat16()), lambda: m.norm_out(y2, k2, i2.long(), 4)):
        with pytest.raises(TypeError):
            f()
    for f in (lambda: m.norm_in(x, w, eps=-1.0), lambda: m.norm_out(y2, k2, gate=w[:4]),
              lambda: m.norm_out(y2, k2, next_out=x)):
        with pytest.raises(m.MoEError):
            f()
