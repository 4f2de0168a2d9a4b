"""Adapters of the experts' down projection on an expert-parallel rank: its slots of other
ranks' experts (ids outside [0, E)) have rows of h and y that no call writes; the adapters
leave them alone, and the layer's partial output is the oracle's."""
import numpy as np
import pytest
import torch

import oracle
from oracle import layer_oracle as lo
from synth import make_inputs
from tests.gpu_util import TOL, moe, say
from tests.layer_util import U, close, f64, gen, rand

pytestmark = pytest.mark.gpu
EPS = 1e-6


def expert_slots(adapter, ids, E):
    """What lora_add's lists are made of: adapter * E + expert of the slots served here."""
    away = (adapter < 0) | (ids < 0) | (ids >= E)
    return torch.where(away, -1, adapter * E + ids).int()


@pytest.mark.parametrize("dtype,block_m", [("bf16", 16), ("bf16", 64), ("fp8", 64), ("fp8", 256)])
@pytest.mark.parametrize("rank", [0, 1, 3])
def test_adapters_on_an_expert_parallel_rank(dtype, block_m, rank):
    T, E, H, I, k, G, adapters, r = 24, 16, 256, 256, 4, 4, 3, 8
    say(f"adapters on rank {rank} of {G}: {dtype} block_m={block_m}")
    m, g, El = moe(), gen(rank), 16 // 4
    inp = make_inputs(T, E, H, I, k, dtype=dtype, routing="normal", seed=3, device="cuda")
    here = slice(rank * El, (rank + 1) * El)
    ids, w = m.route_topk(inp.logits, k)
    ids = (ids - rank * El).contiguous()
    lists = m.align_block(ids, El, block_m)
    code = m.MOE_DTYPE_BF16 if dtype == "bf16" else m.MOE_DTYPE_FP8
    ws = m.alloc_workspace(T, El, H, I, k, block_m, code, "cuda")
    h, y = m.ffn_intermediates(ws, T, El, H, I, k, block_m, code)
    h.fill_(float("nan"))
    y.fill_(77.0)
    args = (ids, w, *lists, block_m, m.STAGE_PREP | m.STAGE_FC1 | m.STAGE_FC2, ws)
    if dtype == "bf16":
        m.ffn_bf16(inp.x, inp.w1[here], inp.w2[here], *args)
    else:
        m.ffn_fp8(inp.x, inp.w1[here], inp.w1_scale[here], inp.w2[here], inp.w2_scale[here], *args)
    n = adapters * El
    adapter = torch.randint(-1, adapters, (T, 1), generator=g).cuda()
    a = rand(g, n, r, I, dtype="bf16", std=I ** -0.5)
    b, scale = rand(g, n, H, r, dtype="bf16", std=r ** -0.5), rand(g, n)
    slots = expert_slots(adapter, ids, El)
    before = y.clone()
    m.lora_add(y, h, a, b, *m.align_block(slots, n, block_m), block_m, scale=scale)
    res, nw = rand(g, T, H, dtype="bf16"), rand(g, H)
    out, nxt = m.norm_out(y, w, ids, El, residual=res, next_weight=nw, eps=EPS,
                          dtype=torch.bfloat16)
    torch.cuda.synchronize()
    away = ((ids < 0) | (ids >= El)).view(-1)
    assert bool(away.any()) and not bool(away.all())
    assert bool((y[away] == 77).all()) and bool(torch.isnan(h[away]).all())
    # rows of the rank's own experts: the adapter's term on the GPU's own h and y
    flat = slots.view(-1).cpu().numpy()
    hh = np.nan_to_num(f64(h))
    ref = lo.lora_add(f64(before), hh, f64(a), f64(b), flat, f64(scale))
    assert oracle.normwise_rel_err(f64(y)[~away.cpu().numpy()],
                                   ref[~away.cpu().numpy()]) <= TOL["bf16"]
    ref_out, ref_next = lo.norm_out(ref, f64(w), ids.cpu().numpy(), El, residual=f64(res),
                                    next_weight=f64(nw), eps=EPS)
    assert oracle.normwise_rel_err(f64(out), ref_out) <= TOL["bf16"]
    assert oracle.normwise_rel_err(f64(nxt), ref_next) <= TOL["bf16"]


@pytest.mark.parametrize("r", [8, 40])
def test_more_adapters_than_a_call_takes(r):
    say(f"adapters split over two calls, r={r}")
    m, g = moe(), gen(r)
    S, n, K, N, M = 200, 1500, 72, 136, 64
    ids = torch.randint(-1, n, (S, 1), generator=g).int().cuda()
    x, y = rand(g, S, K, dtype="bf16"), rand(g, S, N, dtype="bf16")
    a, b = rand(g, n, r, K, dtype="bf16"), rand(g, n, N, r, dtype="bf16")
    with pytest.raises(m.MoEError):
        m.align_block(ids, n, M)
    out = y.clone()
    for first in (0, 1024):
        part = slice(first, min(first + 1024, n))
        count = part.stop - first
        mine = (ids >= first) & (ids < part.stop)
        lists = m.align_block(torch.where(mine, ids - first, -1).int(), count, M)
        m.lora_add(out, x, a[part], b[part], *lists, M)
    torch.cuda.synchronize()
    ref = lo.lora_add(f64(y), f64(x), f64(a), f64(b), ids.view(-1).cpu().numpy())
    mag = lo.lora_add(np.zeros((S, N)), np.abs(f64(x)), np.abs(f64(a)), np.abs(f64(b)),
                      ids.view(-1).cpu().numpy())
    close(out, ref, (K + r + 8) * U * mag + U * np.abs(f64(y)), "bf16", "out")
