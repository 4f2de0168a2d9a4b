"""GPU parity of the router projection against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo
from tests.gpu_util import moe, say
from tests.layer_util import U, f64, gen, rand, sentinel

pytestmark = pytest.mark.gpu


def _check(x, w, bias, got):
    xd, wd = f64(x), f64(w)
    ref = lo.router_logits(xd, wd, None if bias is None else f64(bias))
    # fp32 sums of H exact products (bf16), or products kept to 2^-23 (fp32), in any order
    tol = (x.shape[1] + 3) * U * (np.abs(xd) @ np.abs(wd).T)
    if bias is not None:
        tol = tol + U * np.abs(ref)
    err = np.abs(f64(got) - ref)
    # and near the size a sum of independent roundings has
    rms = np.sqrt(np.mean(err ** 2)) / np.sqrt(np.mean((np.linalg.norm(xd, axis=1)[:, None]
                                                        * np.linalg.norm(wd, axis=1)) ** 2))
    print(f"    largest error {np.max(err / (tol + 1e-37)):.4f} of its bound, "
          f"rms {rms / U:.2f} u |x||w|", flush=True)
    assert np.all(err <= tol + 1e-37)
    assert rms <= 2 * np.sqrt(x.shape[1]) * U


SHAPES = [(1, 1, 8), (1, 8, 256), (3, 5, 16), (16, 64, 4096), (17, 65, 264), (31, 33, 1032),
          (64, 128, 7168), (33, 128, 520), (100, 7, 72), (200, 256, 1024), (5, 1024, 136),
          (129, 300, 2056), (1, 128, 16392), (300, 60, 2048), (1030, 96, 512),
          # 8-row tiles, 16-row tiles and tiles of 32 tokens, on both sides of their limits
          (95 * 16, 16, 136), (95 * 16 + 1, 16, 136), (95 * 32, 64, 72), (95 * 32 + 1, 33, 200),
          (2040, 128, 1032), (4100, 70, 264), (1000, 1000, 64),
          # every tile on both sides of the sizes from which a CU gets one more
          (2048, 8, 72), (2049, 8, 72), (520, 130, 200), (1024, 128, 136), (1025, 128, 264),
          (2048, 128, 72), (2049, 97, 136), (4096, 20, 520), (4100, 33, 136), (8200, 64, 72),
          (4097, 128, 1032)]


@pytest.mark.parametrize("T,E,H", SHAPES)
@pytest.mark.parametrize("dtypes", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_router_parity(T, E, H, dtypes):
    say(f"router T={T} E={E} H={H} {dtypes}")
    g = gen(T + E + H)
    x, w = rand(g, T, H, dtype=dtypes[0]), rand(g, E, H, dtype=dtypes[1])
    bias = rand(g, E)
    out, intact = sentinel((T, E), "f32")
    moe().router_logits(x, w, bias, out=out)
    torch.cuda.synchronize()
    intact()
    _check(x, w, bias, out)
    again = moe().router_logits(x, w, bias)
    assert torch.equal(out, again)                        # the same bits
    _check(x, w, None, moe().router_logits(x, w))


@pytest.mark.parametrize("T", [5, 300, 4100])
def test_router_logits_off_the_16_byte_grid(T):
    say(f"router T={T}: logits 4 bytes off")
    g = gen(T)
    x, w, bias = rand(g, T, 72, dtype="bf16"), rand(g, 64, 72, dtype="bf16"), rand(g, 64)
    buf = torch.full((T * 64 + 8,), 12345.0, device="cuda")
    out = buf[1:1 + T * 64].view(T, 64)
    assert out.data_ptr() % 16 == 4
    moe().router_logits(x, w, bias, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, moe().router_logits(x, w, bias))
    assert float(buf[0]) == 12345.0 and bool((buf[1 + T * 64:] == 12345.0).all())


def test_router_wide_range():
    # magnitudes from 2^-60 to 2^60 in one row: every product counts at its own size
    say("router: wide range")
    g = gen(5)
    for xd, wd in (("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")):
        scale = torch.exp2(torch.linspace(-60, 60, 256))
        x = (torch.randn(4, 256, generator=g) * scale).to(torch.float32)
        w = (torch.randn(9, 256, generator=g) / scale).to(torch.float32)
        x = x.bfloat16().cuda() if xd == "bf16" else x.cuda()
        w = w.bfloat16().cuda() if wd == "bf16" else w.cuda()
        got = moe().router_logits(x, w)
        ref = lo.router_logits(f64(x), f64(w))
        tol = (256 + 3) * U * (np.abs(f64(x)) @ np.abs(f64(w)).T)
        assert np.all(np.abs(f64(got) - ref) <= tol)


def test_router_non_finite_stay_in_their_rows():
    say("router: infinities and NaN")
    g = gen(6)
    x, w = rand(g, 40, 264, dtype="bf16"), rand(g, 33, 264, dtype="f32")
    ref = moe().router_logits(x, w)
    x[3, 5] = float("nan")
    x[20, 100] = float("inf")
    w[7, 200] = float("inf")
    got = moe().router_logits(x, w)
    bad = torch.zeros((40, 33), dtype=torch.bool, device="cuda")
    bad[3] = bad[20] = True
    bad[:, 7] = True
    assert not bool(torch.isfinite(got[bad]).any())
    assert torch.equal(got[~bad], ref[~bad])


def test_router_empty_batch_and_checks():
    say("router: T=0, binding checks")
    m = moe()
    x, w = (torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda"),
            torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda"))
    assert m.router_logits(x[:0], w).shape == (0, 8)
    for f in (lambda: m.router_logits(x, w[:, :32].contiguous()), lambda: m.router_logits(x, w.t()),
              lambda: m.router_logits(x, w, bias=torch.zeros(7, device="cuda")),
              lambda: m.router_logits(x, w.cpu()),
              lambda: m.router_logits(x, w, out=torch.zeros((4, 9), device="cuda"))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(m.MoEError):
        m.router_logits(x.float(), w)


def test_router_rows_past_32_bit_offsets():
    T, H = 270000, 8192
    say(f"router T={T} H={H}")
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 2 ** 31
    x[-1, :] = 1
    x[5, 3] = 2
    w = torch.ones((4, H), dtype=torch.bfloat16, device="cuda")
    got = moe().router_logits(x, w)
    torch.cuda.synchronize()
    assert bool((got[-1] == H).all()) and bool((got[5] == 2).all())
    got[-1] = got[5] = 0
    assert not bool(got.any())
