"""The exact inputs of the router projection's tests see a lost plane: the same arithmetic on
the CPU meets them in 24 bits and misses them in 16 or 8 (no GPU needed)."""
import pytest
import torch

from tests.exact_util import (RMS_LIMIT, exactly, rms_error, router_emulated, router_exact,
                              router_sizes)

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("x_dtype,kind", [(F32, "w"), (F32, "x"), (F32, "rest"), (BF16, "w"),
                                          (BF16, "rest")])
def test_router_exact_sees_lost_planes(x_dtype, kind):
    t = router_exact(torch.Generator().manual_seed(1), 20, 17, 136, x_dtype, kind)
    assert torch.equal(router_emulated(t).double(), t["ref"])
    lost = "x_planes" if kind == "x" else "w_planes"
    for count in (1, 2):
        got = router_emulated(t, **{lost: count})
        assert not bool((got.double() == t["ref"]).any())
        assert not exactly(got, t["ref"], t["off"])


@pytest.mark.parametrize("H", [64, 136, 1032, 4096])
@pytest.mark.parametrize("x_dtype", [F32, BF16])
def test_router_rms_limit_sees_lost_planes(H, x_dtype):
    g = torch.Generator().manual_seed(H)
    t = dict(x=torch.randn(64, H, generator=g).to(x_dtype), w=torch.randn(64, H, generator=g))
    ref = t["x"].double() @ t["w"].double().t()
    sizes = router_sizes(t["x"].double(), t["w"].double())
    assert rms_error(router_emulated(t), ref, sizes) <= RMS_LIMIT
    assert rms_error(t["x"].float() @ t["w"].t(), ref, sizes) <= RMS_LIMIT
    assert rms_error(router_emulated(t, w_planes=2), ref, sizes) > RMS_LIMIT
    if x_dtype == F32:
        assert rms_error(router_emulated(t, x_planes=2), ref, sizes) > RMS_LIMIT
