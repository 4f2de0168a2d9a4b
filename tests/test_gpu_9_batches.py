"""One row in batches of different sizes and company: at equal sizes its bits do not change
with the other rows; at other sizes (other kernels, slices, orders of sums) every result stays
within the fp32 bound of its own."""
import pytest
import torch

from tests.gpu_util import moe, say
from tests.layer_util import gen, rand
from tests.test_gpu_9_lora import _check as check_lora
from tests.test_gpu_9_norms import _check_in, _check_out, _args_out
from tests.test_gpu_9_router import _check as check_router

pytestmark = pytest.mark.gpu
EPS = 1e-5


def _adapters(g, n, r, K, N):
    return dict(a=rand(g, n, r, K, dtype="bf16", std=K ** -0.5), b=rand(g, n, N, r, dtype="bf16"),
                scale=rand(g, n))


# sizes on both sides of the rules: one launch or two, by row or shared b, slices, 16 or 32 rows
@pytest.mark.parametrize("n,r,K,N,sizes", [
    (1, 16, 1032, 136, (1, 2, 7, 8, 9)), (16, 64, 520, 264, (16, 31, 32, 127, 128)),
    (3, 128, 2056, 136, (3, 23, 24, 96, 300)), (40, 24, 264, 200, (39, 319, 320, 1300)),
    (2, 8, 520, 72, (15, 16, 64, 4095, 4096))])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_lora_row_in_batches(n, r, K, N, sizes, dt):
    m, g = moe(), gen(n + r + K)
    f = _adapters(g, n, r, K, N)
    row_x, row_y = rand(g, 1, K, dtype=dt), rand(g, 1, N, dtype=dt)
    for S in sizes:
        say(f"lora row in a batch of {S}, n={n} r={r} {dt}")
        got = []
        for at in (0, S // 2, S - 1):
            d = dict(f, x=rand(g, S, K, dtype=dt), y=rand(g, S, N, dtype=dt),
                     ids=torch.randint(-1, n, (S, 1), generator=g).int().cuda())
            d["x"][at], d["y"][at], d["ids"][at] = row_x[0], row_y[0], 0
            plan = m.align_block(d["ids"], n, 64)
            out = m.lora_add(d["y"], d["x"], d["a"], d["b"], *plan, 64, scale=d["scale"],
                             out=d["y"].clone())
            if at == 0:
                check_lora(d, out, d["y"])
            got.append(out[at].clone())
        assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("E,H", [(8, 264), (60, 1032), (128, 520)])
@pytest.mark.parametrize("dtypes", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_router_row_in_batches(E, H, dtypes):
    m, g = moe(), gen(E + H)
    row, w, bias = rand(g, 1, H, dtype=dtypes[0]), rand(g, E, H, dtype=dtypes[1]), rand(g, E)
    for T in (1, 9, 64, 1030, 2100, 4100):
        say(f"router row in a batch of {T}, E={E} H={H} {dtypes}")
        got = []
        for at in (0, T // 2, T - 1):
            x = rand(g, T, H, dtype=dtypes[0])
            x[at] = row[0]
            out = m.router_logits(x, w, bias)
            got.append(out[at].clone())
        check_router(row, w, bias, got[0].view(1, E))
        assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("H,dt", [(4360, "bf16"), (1032, "bf16"), (2300, "f32")])
def test_norm_rows_in_batches(H, dt):
    m, g = moe(), gen(H)
    row, w = rand(g, 1, H, dtype=dt), rand(g, H)
    one = _args_out(1, 3, H, dt, dt, 5)
    for T in (1, 5, 511, 512, 900):
        say(f"norm rows in a batch of {T}, H={H} {dt}")
        got, out = [], []
        for at in (0, T // 2, T - 1):
            x = rand(g, T, H, dtype=dt)
            x[at] = row[0]
            got.append(m.norm_in(x, w, eps=EPS)[0][at].clone())
            a = _args_out(T, 3, H, dt, dt, T + at)
            a["weight"], a["next_weight"] = one["weight"], one["next_weight"]
            a["y"][3 * at:3 * at + 3] = one["y"]
            for name in ("topk_ids", "topk_weights", "shared", "gate", "residual"):
                a[name][at] = one[name][0]
            o, nxt = m.norm_out(**a, scale=0.5, eps=EPS)
            out.append((o[at].clone(), nxt[at].clone()))
        _check_in(row, None, w, 1.0, got[0].view(1, H), None, dt)
        _check_out(one, 0.5, out[0][0].view(1, H), out[0][1].view(1, H), dt)
        for q in (1, 2):
            assert torch.equal(got[0], got[q])
            assert torch.equal(out[0][0], out[q][0]) and torch.equal(out[0][1], out[q][1])
