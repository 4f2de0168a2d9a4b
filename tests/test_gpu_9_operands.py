"""The operators around the FFN on operands that lie next to each other in one allocation:
refusing overlaps does not refuse neighbours, and nothing is written beside an output."""
import pytest
import torch

from tests.gpu_util import moe, say
from tests.layer_util import gen, rand

pytestmark = pytest.mark.gpu


def packed(**tensors):
    """The tensors' values in one buffer, one right after the other (each a multiple of 16
    bytes); the buffer, and views of it by name."""
    sizes = {n: t.numel() * t.element_size() for n, t in tensors.items()}
    assert all(s % 16 == 0 for s in sizes.values()), sizes
    buf = torch.empty(sum(sizes.values()), dtype=torch.uint8, device="cuda")
    views, at = {}, 0
    for n, t in tensors.items():
        views[n] = buf[at:at + sizes[n]].view(t.dtype).view(t.shape)
        views[n].copy_(t)
        at += sizes[n]
    return buf, views


def only_written(buf, views, names, call):
    """Runs call and checks that of the buffer the named views alone have changed."""
    before = {n: t.clone() for n, t in views.items()}
    call()
    torch.cuda.synchronize()
    for n, t in views.items():
        if n not in names:
            assert torch.equal(t, before[n]), n


def test_norms_between_their_operands():
    say("norms: operands in a row")
    m, g = moe(), gen(1)
    T, k, H = 12, 2, 264
    x, res, w = rand(g, T, H, dtype="bf16"), rand(g, T, H, dtype="bf16"), rand(g, H)
    buf, v = packed(x=x, out=x, w=w, s=x, res=res)
    only_written(buf, v, ("out", "s"), lambda: m.norm_in(
        v["x"], v["w"], v["res"], 0.5, out=v["out"], residual_out=v["s"]))
    ref, s = m.norm_in(x, w, res, 0.5)
    assert torch.equal(v["out"], ref) and torch.equal(v["s"], s)

    y, nw = rand(g, T * k, H, dtype="bf16"), rand(g, H)
    wts = torch.rand((T, k), generator=g).cuda()
    ids = torch.randint(-1, 6, (T, k), generator=g).int().cuda()
    gate = rand(g, T)
    buf, v = packed(wts=wts, out=x, ids=ids, w=w, nxt=x, nw=nw, y=y, gate=gate, sh=x, res=res)
    only_written(buf, v, ("out", "nxt"), lambda: m.norm_out(
        v["y"], v["wts"], v["ids"], 5, v["sh"], v["gate"], v["res"], v["w"], v["nw"],
        out=v["out"], next_out=v["nxt"]))
    ref, nxt = m.norm_out(y, wts, ids, 5, x, gate, res, w, nw)
    assert torch.equal(v["out"], ref) and torch.equal(v["nxt"], nxt)


def test_router_between_its_operands():
    say("router: operands in a row")
    m, g = moe(), gen(2)
    x, w, bias = rand(g, 12, 136, dtype="bf16"), rand(g, 20, 136, dtype="bf16"), rand(g, 20)
    buf, v = packed(x=x, bias=bias, out=torch.zeros((12, 20)).cuda(), w=w)
    only_written(buf, v, ("out",),
                 lambda: m.router_logits(v["x"], v["w"], v["bias"], out=v["out"]))
    assert torch.equal(v["out"], m.router_logits(x, w, bias))


@pytest.mark.parametrize("S,r", [(12, 16), (12, 40), (64, 16), (64, 72)])
def test_lora_between_its_operands(S, r):
    say(f"lora: operands in a row S={S} r={r}")
    m, g = moe(), gen(3)
    n, K, N, M = 4, 136, 264, 16
    ids = torch.randint(-1, n, (S, 1), generator=g).int().cuda()
    sid, ba, npad = m.align_block(ids, n, M)
    x, y = rand(g, S, K, dtype="bf16"), rand(g, S, N, dtype="bf16")
    a, b = rand(g, n, r, K, dtype="bf16"), rand(g, n, N, r, dtype="bf16")
    scale = rand(g, n)
    ref = m.lora_add(y, x, a, b, sid, ba, npad, M, scale=scale, out=y.clone())
    fit = lambda t: torch.cat([t, t.new_zeros(-t.numel() % 4)])  # noqa: E731
    ws = torch.zeros(m.lora_workspace_bytes(S, n, K, r, M), dtype=torch.uint8, device="cuda")
    buf, v = packed(ws=ws, x=x, a=a, out=y, b=b, sid=fit(sid), ba=fit(ba), npad=fit(npad), y=y,
                    scale=scale)
    call = lambda out: m.lora_add(v["y"], v["x"], v["a"], v["b"], v["sid"], v["ba"],  # noqa: E731
                                  v["npad"], M, scale=v["scale"], out=out, workspace=v["ws"])
    only_written(buf, v, ("out", "ws"), lambda: call(v["out"]))
    assert torch.equal(v["out"], ref)
    only_written(buf, v, ("y", "ws"), lambda: call(None))      # in place
    assert torch.equal(v["y"], ref)
    # slices of one matrix's columns, with the factors right behind its last row
    wide = torch.full((S, 3 * N), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 2 * N:] = y
    buf, v2 = packed(wide=wide, a=a, b=b)
    m.lora_add(v2["wide"][:, 2 * N:], x, v2["a"], v2["b"], sid, ba, npad, M, scale=scale,
               out=v2["wide"][:, :N])
    torch.cuda.synchronize()
    live = (ids.view(-1) >= 0).nonzero().view(-1)
    assert torch.equal(v2["wide"][live][:, :N], ref[live])
    assert bool((v2["wide"][:, N:2 * N] == 5).all()) and torch.equal(v2["wide"][:, 2 * N:], y)
    assert torch.equal(v2["a"], a) and torch.equal(v2["b"], b)
