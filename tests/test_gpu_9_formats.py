"""The intermediates of every weight format's workspace, as ffn_intermediates shows them: h and
y against the oracle's arithmetic, the adapters and the combine on them."""
import numpy as np
import pytest
import torch

import oracle
from oracle import layer_oracle as lo
from synth import make_inputs
from tests.gpu_util import TOL, moe, say
from tests.layer_util import close, f64, gen, rand
from tests.test_gpu_9_lora import _check as check_lora

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _weights(inp, name, E):
    """The experts' weights as fp64 values."""
    host = {"w1": (inp.host_w1, inp.host_w1_scale), "w2": (inp.host_w2, inp.host_w2_scale)}[name]
    if inp.dtype == "fp8_block":
        return [oracle.dequant_blocks(host[0](e), host[1]()[e]) for e in range(E)]
    if inp.dtype == "fp8":
        return [oracle.e4m3fn_decode(host[0](e)) * host[1]()[e][:, None] for e in range(E)]
    return [oracle.bf16_bits_to_f64(host[0](e)) for e in range(E)]


CASES = [("w8a16", 24, 8, 256, 384, 3), ("w8a16", 5, 4, 128, 256, 2), ("w8a16", 90, 4, 512, 256, 2),
         ("fp8_block", 24, 8, 256, 384, 3), ("fp8_block", 90, 4, 512, 256, 2),
         ("fp8", 9, 8, 200, 136, 3), ("fp8", 90, 4, 512, 256, 2), ("bf16", 9, 8, 200, 136, 3),
         ("bf16", 90, 4, 512, 256, 2)]


@pytest.mark.parametrize("block_m", [16, 64, 256])
@pytest.mark.parametrize("fmt,T,E,H,I,k", CASES)
def test_intermediates_of_every_format(fmt, T, E, H, I, k, block_m):
    say(f"intermediates {fmt} T={T} E={E} H={H} I={I} k={k} block_m={block_m}")
    m, g = moe(), gen(T + H)
    inp = make_inputs(T, E, H, I, k, dtype="fp8" if fmt == "w8a16" else fmt, routing="normal",
                      seed=T + block_m, device="cuda")
    code = {"w8a16": m.MOE_DTYPE_W8A16, "fp8": m.MOE_DTYPE_FP8, "bf16": m.MOE_DTYPE_BF16,
            "fp8_block": m.MOE_DTYPE_FP8_BLOCK}[fmt]
    ids, w, *lists = m.route_align(inp.logits, k, block_m)
    ws = m.alloc_workspace(T, E, H, I, k, block_m, code, "cuda")
    args = (ids, w, *lists, block_m, m.STAGE_PREP | m.STAGE_FC1 | m.STAGE_FC2, ws)
    if fmt == "bf16":
        m.ffn_bf16(inp.x, inp.w1, inp.w2, *args)
    else:
        call = {"w8a16": m.ffn_w8a16, "fp8": m.ffn_fp8, "fp8_block": m.ffn_fp8_block}[fmt]
        call(inp.x, inp.w1, inp.w1_scale, inp.w2, inp.w2_scale, *args)
    h, y = m.ffn_intermediates(ws, T, E, H, I, k, block_m, code)
    torch.cuda.synchronize()
    tol = TOL["fp8"] if "fp8" in fmt else TOL["bf16"]
    w1, w2 = _weights(inp, "w1", E), _weights(inp, "w2", E)
    x, e_of = oracle.bf16_bits_to_f64(inp.host_x()), ids.view(-1).cpu().numpy()
    href = np.zeros((T * k, I))
    for s in range(T * k):
        gu = w1[e_of[s]] @ x[s // k]
        href[s] = gu[:I] / (1 + np.exp(-gu[:I])) * gu[I:]
    yref = np.stack([w2[e_of[s]] @ f64(h)[s] for s in range(T * k)])   # of the GPU's own h
    assert oracle.normwise_rel_err(f64(h), href) <= tol
    assert oracle.normwise_rel_err(f64(y), yref) <= tol

    # the adapters on them, to their own bound, and the combine
    adapters, r = 2, 16
    n = adapters * E
    adapter = torch.randint(-1, adapters, (T, 1), generator=g).cuda()
    slots = torch.where(adapter < 0, -1, adapter * E + ids).int()
    d = dict(x=h, a=rand(g, n, r, I, dtype="bf16", std=I ** -0.5),
             b=rand(g, n, H, r, dtype="bf16", std=r ** -0.5), scale=rand(g, n),
             ids=slots.view(-1, 1), y=y)
    before = y.clone()
    m.lora_add(y, h, d["a"], d["b"], *m.align_block(slots, n, block_m), block_m,
               scale=d["scale"])
    torch.cuda.synchronize()
    check_lora(d, y, before)
    out, _ = m.norm_out(y, w, ids, E, dtype=torch.bfloat16)
    ref, _ = lo.norm_out(f64(y), f64(w), ids.cpu().numpy(), E)
    mag, _ = lo.norm_out(np.abs(f64(y)), f64(w), ids.cpu().numpy(), E)
    close(out, ref, (k + 8) * 2.0 ** -24 * mag, "bf16", "combine")
