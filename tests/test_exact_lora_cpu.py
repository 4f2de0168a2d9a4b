"""The exact inputs of the adapters' tests see a lost plane: the same
arithmetic on the CPU meets them in 24 bits and misses them in 16 or 8 (no GPU needed)."""
import pytest
import torch

from tests.exact_util import (RMS_LIMIT, cut, exactly, full_floats, lora_emulated, lora_exact,
                              lora_sizes, planes, rms_error)

BF16, F32 = torch.bfloat16, torch.float32


def test_planes_are_the_value():
    v = full_floats(torch.Generator().manual_seed(0), 4096)
    p = planes(v)
    assert torch.equal(p[0] + p[1] + p[2], v) and torch.equal(cut(v, 3), v)
    assert bool((p[2] != 0).all()) and not bool((cut(v, 2) == v).any())
    assert all(torch.equal(q, q.bfloat16().float()) for q in p)


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("x_dtype,y_dtype", [(BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("r", [8, 24, 64, 256])
def test_lora_exact_sees_lost_planes(r, x_dtype, y_dtype, whole):
    t = lora_exact(torch.Generator().manual_seed(r), 9, 3, r, 3 * r // 2 + 40, 136, x_dtype, whole)
    ref = t["d"].float().to(y_dtype)
    assert torch.equal(lora_emulated(t, y_dtype), ref) and exactly(ref, t["d"], t["off"])
    live = t["ids"] >= 0
    cuts = [dict(z_planes=2), dict(z_planes=1)]
    if x_dtype == F32:
        cuts += [dict(x_planes=2), dict(x_planes=1)]
    for c in cuts:
        got = lora_emulated(t, y_dtype, **c)
        # rounded to bf16 the whole of v shows little of its low planes; what is left after
        # the others are taken away shows them all
        if y_dtype == F32 or not whole:
            assert not bool((got[live] == ref[live]).any()), c
            assert not exactly(got, t["d"], t["off"]), c


@pytest.mark.parametrize("r,K", [(8, 64), (16, 520), (64, 1032), (256, 2048)])
def test_lora_rms_limit_sees_lost_planes(r, K):
    g = torch.Generator().manual_seed(r)
    S, N = 24, 136
    t = dict(x=torch.randn(S, K, generator=g), a=(torch.randn(1, r, K, generator=g) * K ** -0.5)
             .bfloat16(), b=torch.randn(1, N, r, generator=g).bfloat16(), scale=torch.ones(1),
             ids=torch.zeros(S, dtype=torch.long))
    z = t["x"].double() @ t["a"][0].double().t()
    ref = z @ t["b"][0].double().t()
    sizes = lora_sizes(t["x"].double(), t["a"][0].double(), t["b"][0].double())
    assert rms_error(lora_emulated(t, F32), ref, sizes) <= RMS_LIMIT
    plain = (t["x"] @ t["a"][0].float().t()) @ t["b"][0].float().t()
    assert rms_error(plain, ref, sizes) <= RMS_LIMIT
    for c in (dict(x_planes=2), dict(z_planes=2)):
        assert rms_error(lora_emulated(t, F32, **c), ref, sizes) > RMS_LIMIT, c
