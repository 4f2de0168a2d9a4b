"""Exact results of the adapters on the GPU: no bit of fp32 rows or of the rank-r intermediate
is lost, whichever kernels the sizes choose; and the rms error of random fp32 rows."""
import pytest
import torch

from tests.exact_util import RMS_LIMIT, exactly, lora_exact, lora_sizes, rms_error
from tests.gpu_util import moe, say
from tests.layer_util import DT, gen, rand

pytestmark = pytest.mark.gpu

LORA = [  # S, n, r, K, N, block_m
    # one launch, r 8 to 32
    (7, 5, 8, 136, 136, 64), (7, 5, 16, 4104, 136, 16), (7, 5, 24, 136, 200, 64),
    (7, 5, 32, 136, 136, 4),
    # shrink and expansion by columns
    (600, 513, 8, 72, 72, 64), (300, 260, 16, 72, 136, 64), (300, 171, 24, 72, 72, 64),
    (200, 129, 32, 1032, 72, 64),
    # expansion row by row, few and many slices of K
    (7, 5, 64, 136, 136, 64), (9, 9, 40, 1032, 200, 2), (7, 5, 128, 4104, 264, 64),
    (7, 5, 256, 520, 136, 16),
    # b shared between rows; 16 ranks to a workgroup of the shrink, or more
    (64, 3, 8, 136, 136, 64), (64, 3, 16, 136, 136, 16), (64, 3, 24, 4104, 264, 64),
    (64, 3, 64, 136, 136, 64), (64, 3, 128, 264, 136, 64), (64, 3, 256, 1032, 136, 64),
    (1000, 9, 96, 200, 136, 64), (300, 3, 248, 520, 264, 32),
    (64, 4, 64, 4096, 136, 64), (128, 16, 24, 4096, 136, 64), (100, 4, 128, 2048, 136, 64),
    # 32 rows at a time in the shrink
    (4100, 2, 64, 136, 136, 64), (4100, 3, 16, 200, 136, 32), (4100, 2, 24, 136, 72, 256),
    (4200, 1, 160, 264, 72, 64)]


@pytest.mark.parametrize("S,n,r,K,N,block_m", LORA)
@pytest.mark.parametrize("xdt,ydt", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"),
                                     ("f32", "f32")])
@pytest.mark.parametrize("whole", [False, True], ids=["rest", "whole"])
def test_lora_exact(S, n, r, K, N, block_m, xdt, ydt, whole):
    say(f"lora exact S={S} n={n} r={r} K={K} N={N} M={block_m} {xdt}->{ydt} whole={whole}")
    m = moe()
    t = lora_exact(gen(S + r + K), S, n, r, K, N, DT[xdt], whole)
    plan = m.align_block(t["ids"].int().view(S, 1).cuda(), n, block_m)
    y = torch.zeros((S, N), dtype=DT[ydt], device="cuda")
    out = m.lora_add(y, t["x"].cuda(), t["a"].cuda(), t["b"].cuda(), *plan, block_m,
                     scale=t["scale"].cuda())
    assert exactly(out.cpu(), t["d"], t["off"])


@pytest.mark.parametrize("S,n,r,K,N", [(7, 5, 16, 1024, 264), (300, 260, 16, 520, 136),
                                       (7, 5, 64, 1024, 264), (64, 3, 16, 1024, 264),
                                       (64, 3, 64, 520, 264), (64, 3, 256, 1024, 136),
                                       (4100, 2, 64, 264, 136)])
def test_lora_rms_error(S, n, r, K, N):
    say(f"lora rms S={S} n={n} r={r} K={K} N={N}")
    m, g = moe(), gen(S + r + K)
    ids = torch.arange(S) % n
    x, a = rand(g, S, K), rand(g, n, r, K, dtype="bf16", std=K ** -0.5)
    b, y = rand(g, n, N, r, dtype="bf16"), torch.zeros((S, N), device="cuda")
    plan = m.align_block(ids.int().view(S, 1).cuda(), n, 64)
    got = m.lora_add(y, x, a, b, *plan, 64).cpu()
    x, a, b = x.double().cpu(), a.double().cpu(), b.double().cpu()
    ref, sizes = torch.zeros(S, N).double(), torch.zeros(S, N).double()
    for q in range(n):
        ref[ids == q] = (x[ids == q] @ a[q].t()) @ b[q].t()
        sizes[ids == q] = lora_sizes(x[ids == q], a[q], b[q])
    rms = rms_error(got, ref, sizes)
    print(f"    rms error {rms:.2f}, limit {RMS_LIMIT}", flush=True)
    assert rms <= RMS_LIMIT
