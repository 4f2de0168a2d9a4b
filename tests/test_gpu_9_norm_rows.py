"""The norms at the row lengths where the number of waves and of vectors to a thread changes."""
import pytest
import torch

from tests.gpu_util import moe, say
from tests.layer_util import gen, rand
from tests.test_gpu_9_norms import _args_out, _check_in, _check_out

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.mark.parametrize("T", [1, 3, 600])
@pytest.mark.parametrize("H,ydt,dt", [
    (2048, "bf16", "bf16"), (4096, "bf16", "bf16"), (4104, "bf16", "bf16"),
    (8192, "bf16", "bf16"), (8200, "bf16", "f32"), (2048, "f32", "bf16"), (2056, "f32", "bf16"),
    (4096, "f32", "bf16"), (4104, "f32", "bf16"), (2048, "f32", "f32"), (2052, "f32", "f32"),
    (4096, "f32", "f32"), (4100, "f32", "f32"), (8196, "f32", "f32")])
def test_norms_at_row_lengths(T, H, ydt, dt):
    say(f"norms T={T} H={H} y {ydt} {dt}")
    g = gen(T + H)
    x, res, w = rand(g, T, H, dtype=dt), rand(g, T, H, dtype=dt, std=3.0), rand(g, H)
    out, s = moe().norm_in(x, w, res, 0.5, EPS)
    _check_in(x, res, w, 0.5, out, s, dt)
    a = _args_out(T, 3, H, ydt, dt, T + H)
    out, nxt = moe().norm_out(**a, scale=0.5, eps=EPS)
    _check_out(a, 0.5, out, nxt, dt)
