"""The operators beside the FFN run together, as a block that trains its own experts and a shared
expert runs them: layer norm, router, routing, dispatch, the experts' products (of the caller: linear
per expert), combine, norm_out with the shared expert; and the gradients on the way back; the same on
a side stream and captured into a graph."""
import numpy as np
import pytest
import torch

import oracle
from oracle import layer_oracle as lo
from tests.gpu_util import moe, say
from tests.layer_util import DT, U, close, f64, gen, rand

pytestmark = pytest.mark.gpu


class Block:
    def __init__(self, T, E, H, I, k, dtype, block_m, seed=0):
        g = gen(seed)
        self.T, self.E, self.H, self.I, self.k, self.block_m, self.dtype = T, E, H, I, k, block_m, dtype
        self.x, self.res = rand(g, T, H, dtype=dtype), rand(g, T, H, dtype=dtype, std=2.0)
        self.gamma, self.beta = 1 + 0.1 * rand(g, H), 0.1 * rand(g, H)
        self.wr = rand(g, E, H, dtype=dtype, std=H ** -0.5)
        self.w1 = rand(g, E, 2 * I, H, dtype=dtype, std=H ** -0.5)
        self.w2 = rand(g, E, H, I, dtype=dtype, std=I ** -0.5)
        self.s1, self.s2 = rand(g, 2 * I, H, dtype=dtype, std=H ** -0.5), rand(
            g, H, I, dtype=dtype, std=I ** -0.5)
        self.b1, self.b2 = 0.1 * rand(g, 2 * I), 0.1 * rand(g, H)
        self.dout = rand(g, T, H, dtype=dtype)

    def experts(self, m, rows, block_expert, n, kw):
        """The expert products of a caller's own: a run of rows at a time."""
        y = torch.zeros_like(rows)
        be = block_expert.tolist()
        for e in range(self.E):
            mine = [b for b, v in enumerate(be) if v == e and b * self.block_m < n]
            if mine:
                a, b = mine[0] * self.block_m, (mine[-1] + 1) * self.block_m
                h = m.linear(rows[a:b], self.w1[e], activation=m.ACT_SILU, gated=True, **kw)
                m.linear(h, self.w2[e], out=y[a:b], **kw)
        return y

    def run(self, stream=None):
        m, kw = moe(), dict(stream=stream)
        u, s = m.layer_norm(self.x, self.gamma, self.beta, self.res, **kw)
        logits = m.router_logits(u, self.wr, **kw)
        ids, w, sid, be, npad = m.route_align(logits, self.k, self.block_m, **kw)
        rows, at = m.dispatch(u, ids, self.E, sid, npad, **kw)
        if stream is not None:
            stream.synchronize()
        n = int(npad)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            y = self.experts(m, rows, be, n, kw)
        h = m.linear(u, self.s1, self.b1, m.ACT_SILU, True, **kw)
        out = m.linear(h, self.s2, self.b2, residual=s, **kw)
        back = m.combine(y, at, w, **kw)
        # and the way back to the layer norm through the dispatched rows
        drows, dw = m.combine_backward(self.dout, y, at, w, sid, npad, **kw)
        dx = m.dispatch_backward(drows, at, **kw)
        grads = m.layer_norm_backward(dx, s, self.gamma, self.dout, **kw)
        return dict(u=u, s=s, ids=ids, w=w, at=at, y=y, back=back, shared=out, drows=drows[:n],
                    dw=dw, dx=dx, dres=grads[1], dgamma=grads[2], dbeta=grads[3], n=n,
                    sid=sid, be=be)


BLOCKS = [(9, 4, 64, 48, 2, "f32", 8), (40, 8, 256, 128, 3, "bf16", 16),
          (1, 8, 72, 40, 2, "bf16", 1), (150, 4, 264, 200, 2, "bf16", 128)]


@pytest.mark.parametrize("T,E,H,I,k,dtype,block_m", BLOCKS)
def test_block_parity(T, E, H, I, k, dtype, block_m):
    say(f"block T={T} E={E} H={H} I={I} k={k} {dtype} block_m={block_m}")
    b = Block(T, E, H, I, k, dtype, block_m)
    got = b.run()
    torch.cuda.synchronize()
    # intermediates are rounded to the type on the way: some ten of them, half a step each, through
    # products of random signs; relative to the largest value
    tol = {"bf16": 16 * 2.0 ** -8, "f32": 1e-4}[dtype]

    def near(name, ref):
        d = np.abs(f64(got[name]) - ref).max() / max(np.abs(ref).max(), 1e-30)
        say(f"    {name}: {d:.2e}")
        assert d <= tol, name

    u, s = lo.layer_norm(f64(b.x), f64(b.gamma), f64(b.beta), f64(b.res))
    near("u", u)
    near("s", s)
    ids, w, at = (got[q].cpu().numpy() for q in ("ids", "w", "at"))
    sid, _, n = oracle.align(ids, E, block_m)
    assert n == got["n"] and np.array_equal(lo.places(sid, n, T * k).reshape(T, k), at)
    y = np.zeros((n, H))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            h = lo.linear(u[t:t + 1], f64(b.w1[e]), act="silu", gated=True)
            y[at[t, j]] = lo.linear(h, f64(b.w2[e]))
    near("back", lo.combine(y, at, w))
    h = lo.linear(u, f64(b.s1), f64(b.b1), "silu", True)
    near("shared", lo.linear(h, f64(b.s2), f64(b.b2), residual=s))
    dout = f64(b.dout)
    drows, dw = lo.combine_backward(dout, y, at, w, n)
    near("drows", drows)
    near("dw", dw)
    dx = lo.combine(drows, at)
    near("dx", dx)
    _, dres, dgamma, dbeta = lo.layer_norm_backward(dx, s, f64(b.gamma), dout)
    near("dres", dres)
    near("dgamma", dgamma)
    near("dbeta", dbeta)


def test_side_stream():
    say("block on a side stream")
    b = Block(*BLOCKS[1])
    ref = b.run()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    got = b.run(stream)
    stream.synchronize()
    for name, t in ref.items():
        if isinstance(t, torch.Tensor):
            assert torch.equal(got[name], t), name


def test_two_at_once():
    """Two blocks on two streams, each with workspaces of its own, give what they give alone; K in
    parts (a workspace) and few rows among them."""
    say("two blocks at once")
    m, g = moe(), gen(5)
    blocks = [Block(*BLOCKS[i], seed=30 + i) for i in (1, 3)]
    xs = [rand(g, T, 4096, dtype="bf16") for T in (100, 200)]
    ws = [rand(g, 512, 4096, dtype="bf16") for _ in xs]
    assert all(m.linear_workspace_bytes(x.shape[0], 512, 4096, False, 1) > 0 for x in xs)

    def both(i, stream):
        return b_run(blocks[i], stream), m.linear(xs[i], ws[i], stream=stream)

    def b_run(b, stream):
        return {n: t for n, t in b.run(stream).items() if isinstance(t, torch.Tensor)}

    ref = [both(i, None) for i in (0, 1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(3):
        # the products of both queued before either is waited for
        got = [[m.linear(xs[i], ws[i], stream=streams[i]) for _ in range(8)] for i in (0, 1)]
        runs = [b_run(blocks[i], streams[i]) for i in (0, 1)]
        torch.cuda.synchronize()
        for i in (0, 1):
            for out in got[i]:
                assert torch.equal(out, ref[i][1])
            for name, t in ref[i][0].items():
                assert torch.equal(runs[i][name], t), name


def test_the_same_expert_twice():
    """A token whose ids name one expert twice has two places, whose rows count twice."""
    say("the same expert twice")
    m, g = moe(), gen(6)
    T, E, H, M = 37, 4, 264, 8
    ids = torch.randint(0, E, (T, 1), generator=g, dtype=torch.int32).cuda().repeat(1, 3)
    ids[:, 2] = (ids[:, 2] + 1) % E
    ids = ids.contiguous()
    x, w = rand(g, T, H), rand(g, T, 3)
    sid, be, n = m.align_block(ids, E, M)
    rows, at = m.dispatch(x, ids, E, sid, n)
    a = at.cpu()
    assert a.unique().numel() == T * 3 and int(a.min()) >= 0
    for j in range(3):
        assert torch.equal(rows[a[:, j].cuda().long()], x)
    close(m.combine(rows, at, w), f64(w).sum(1, keepdims=True) * f64(x),
          4 * U * np.abs(f64(w)).sum(1, keepdims=True) * np.abs(f64(x)), "f32", "combine")
    close(m.dispatch_backward(rows, at), 3 * f64(x), 3 * U * np.abs(f64(x)), "f32", "dx")


def test_with_norm_out():
    """combine is the combine of norm_out on rows in slot order, and the shared expert of linear is
    what norm_out takes."""
    say("combine and linear beside norm_out")
    b = Block(*BLOCKS[1], seed=3)
    m, got = moe(), b.run()
    slots = got["y"][got["at"].long().view(-1)]
    ref, _ = m.norm_out(slots, got["w"], got["ids"], b.E)
    assert torch.equal(got["back"], ref)
    u, s = got["u"], got["s"]
    h = m.linear(u, b.s1, b.b1, m.ACT_SILU, True)
    shared = m.linear(h, b.s2, b.b2)
    one, _ = m.norm_out(slots, got["w"], got["ids"], b.E, shared=shared, residual=s)
    two = m.linear(h, b.s2, b.b2, residual=s.float())
    assert torch.equal(two.bfloat16(), got["shared"])
    # the same three terms, two of them rounded apart
    full = f64(two) + f64(got["back"])
    tol = 2.0 ** -8 * (np.abs(full) + np.abs(f64(shared)) + np.abs(f64(got["back"])))
    assert np.all(np.abs(f64(one) - full) <= 1.01 * tol + 1e-6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graph(dtype):
    """Captured and replayed five times with eager work and synchronisations between; the inputs
    change from replay to replay."""
    say(f"block captured {dtype}")
    m, g = moe(), gen(20)
    T, E, H, I, k, M = 60, 8, 264, 136, 2, 16
    b = Block(T, E, H, I, k, dtype, M, seed=21)
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    sid = torch.empty(m.align_capacity(T, k, E, M), dtype=torch.int32, device="cuda")
    be = torch.empty(sid.numel() // M, dtype=torch.int32, device="cuda")
    npad, w = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    rows = torch.zeros((sid.numel(), H), dtype=DT[dtype], device="cuda")
    drows = torch.zeros_like(rows)
    need = m.linear_workspace_bytes(T, H, I, False, {"bf16": 1, "f32": 0}[dtype])
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    nws = torch.empty(m.layer_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")

    def step():
        u, s = m.layer_norm(b.x, b.gamma, b.beta, b.res)
        m.route_align(m.router_logits(u, b.wr), k, M, out=(ids, w, sid, be, npad))
        _, at = m.dispatch(u, ids, E, sid, npad, out=rows)
        h = m.linear(u, b.s1, b.b1, m.ACT_GELU, True)
        shared = m.linear(h, b.s2, b.b2, residual=s, workspace=ws)
        back = m.combine(rows, at, w)
        _, dw = m.combine_backward(b.dout, rows, at, w, sid, npad, drows=drows)
        dx = m.dispatch_backward(drows, at)
        grads = m.layer_norm_backward(dx, s, b.gamma, b.dout, workspace=nws)
        return [u, s, at, shared, back, dw, dx, *grads]

    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(5):
        b.x.copy_(rand(g, T, H, dtype=dtype))
        b.dout.copy_(rand(g, T, H, dtype=dtype))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in outs] + [rows.clone(), drows.clone()]
        rows.zero_()
        drows.zero_()
        ref = step()
        torch.cuda.synchronize()
        n = int(npad)
        for a, c in zip(kept, ref + [rows, drows]):
            cut = n if a.shape[0] == sid.numel() else a.shape[0]
            assert torch.equal(a[:cut], c[:cut]), i


def test_another_device_or_stream_is_refused():
    m = moe()
    x = torch.zeros((2, 8), device="cuda")
    if torch.cuda.device_count() > 1:
        with torch.cuda.device(1), pytest.raises(ValueError, match="current device"):
            m.layer_norm(x)
    with pytest.raises(ValueError, match="shape"):
        m.layer_norm(x, weight=torch.ones(9, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        m.layer_norm(torch.zeros((8, 16), device="cuda")[:, :8])
    with pytest.raises(ValueError, match="contiguous"):
        m.linear(torch.zeros((8, 16), device="cuda").t(), torch.zeros((4, 8), device="cuda"))
    with pytest.raises(ValueError, match="2 N"):
        m.linear(x, torch.zeros((5, 8), device="cuda"), gated=True)
    with pytest.raises(m.MoEError, match="SHAPE"):
        m.linear(torch.zeros((8, 12), device="cuda"), torch.zeros((4, 12), device="cuda"))
    with pytest.raises(TypeError, match="dtype"):
        m.linear(x, torch.zeros((4, 8), dtype=torch.bfloat16, device="cuda"))
    rows, at = torch.zeros((4, 8), device="cuda"), torch.zeros((2, 2), dtype=torch.int32,
                                                               device="cuda")
    with pytest.raises(TypeError, match="dtype"):
        m.combine(rows, at.long())
    with pytest.raises(ValueError, match="shape"):
        m.combine(rows, at, torch.zeros((2, 3), device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        m.combine_backward(x, rows, at, None, torch.zeros(5, dtype=torch.int32, device="cuda"),
                           torch.zeros(1, dtype=torch.int32, device="cuda"))
