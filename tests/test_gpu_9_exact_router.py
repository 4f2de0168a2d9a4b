"""Exact results of the router projection on the GPU: no bit of an fp32 operand is lost,
whichever tile the sizes choose; and the rms error of random operands."""
import pytest

from tests.exact_util import RMS_LIMIT, exactly, rms_error, router_exact, router_sizes
from tests.gpu_util import moe, say
from tests.layer_util import DT, gen, rand

pytestmark = pytest.mark.gpu

# T, E on every tile: 8 x 8, 16 x 16, 16 x 32 (fp32 w beside bf16 x: 32 x 16), 32 x 32, 32 x 64
# (64 x 32), for the one or other types
ROUTER = [(16, 64), (1024, 128), (1536, 128), (4100, 128), (4096, 8), (2049, 97), (1030, 96)]


@pytest.mark.parametrize("T,E", ROUTER)
@pytest.mark.parametrize("H", [136, 1032])
@pytest.mark.parametrize("xdt,kind", [("f32", "w"), ("f32", "x"), ("f32", "rest"),
                                      ("bf16", "w"), ("bf16", "rest")])
def test_router_exact(T, E, H, xdt, kind):
    say(f"router exact T={T} E={E} H={H} {xdt} {kind}")
    t = router_exact(gen(T + E + H), T, E, H, DT[xdt], kind)
    got = moe().router_logits(t["x"].cuda(), t["w"].cuda())
    assert exactly(got.cpu(), t["ref"], t["off"])


@pytest.mark.parametrize("T,E", ROUTER)
@pytest.mark.parametrize("H", [72, 264, 1024])
@pytest.mark.parametrize("xdt", ["f32", "bf16"])
def test_router_rms_error(T, E, H, xdt):
    say(f"router rms T={T} E={E} H={H} {xdt}")
    g = gen(T + E + H)
    x, w = rand(g, T, H, dtype=xdt), rand(g, E, H)
    got = moe().router_logits(x, w).cpu()
    x, w = x.double().cpu(), w.double().cpu()
    rms = rms_error(got, x @ w.t(), router_sizes(x, w))
    print(f"    rms error {rms:.2f}, limit {RMS_LIMIT}", flush=True)
    assert rms <= RMS_LIMIT
