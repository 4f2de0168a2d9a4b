"""The operators around the FFN run together, as a layer runs them: norm_in,
router_logits, route_align, the FFN's stages with the adapters on its own h and
y, norm_out; the same captured into a graph and replayed, and on a side stream."""
import functools

import numpy as np
import pytest
import torch

import oracle
from oracle import layer_oracle as lo
from synth import make_inputs
from tests.gpu_util import TOL, moe, say
from tests.layer_util import f64, gen, rand

pytestmark = pytest.mark.gpu
EPS = 1e-6


class Layer:
    """One MoE layer with adapters of the experts' down projection."""

    def __init__(self, T, E, H, I, k, dtype, block_m, adapters=3, r=8, seed=0):
        m = moe()
        self.inp = make_inputs(T, E, H, I, k, dtype=dtype, routing="normal", seed=seed,
                               device="cuda")
        g = gen(seed + 1)
        self.T, self.E, self.H, self.I, self.k, self.block_m = T, E, H, I, k, block_m
        self.n = adapters * E
        act = "f32" if dtype == "f32" else "bf16"
        self.x = rand(g, T, H, dtype=act)
        self.res = rand(g, T, H, dtype=act, std=2.0)
        self.shared, self.gate = rand(g, T, H, dtype=act), rand(g, T)
        self.w_in, self.w_out, self.w_next = (1 + 0.1 * rand(g, H) for _ in range(3))
        self.wr = rand(g, E, H, dtype=act, std=H ** -0.5)
        self.bias = rand(g, E, std=0.1)
        self.a = rand(g, self.n, r, I, dtype="bf16", std=I ** -0.5)
        self.b = rand(g, self.n, H, r, dtype="bf16", std=r ** -0.5)
        self.scale = rand(g, self.n)
        # tokens of an adapter each, some of none
        self.adapter = torch.randint(-1, adapters, (T, 1), generator=g).cuda()
        self.code = {"f32": m.MOE_DTYPE_F32, "bf16": m.MOE_DTYPE_BF16, "fp8": m.MOE_DTYPE_FP8}[dtype]
        self.ws = m.alloc_workspace(T, E, H, I, k, block_m, self.code, "cuda")

    def run(self, stream=None):
        m, inp, bm = moe(), self.inp, self.block_m
        kw = dict(stream=stream)
        xn, res = m.norm_in(self.x, self.w_in, self.res, 0.75, EPS, **kw)
        logits = m.router_logits(xn, self.wr, self.bias, **kw)
        ids, w, sid, be, npad = m.route_align(logits, self.k, bm, **kw)
        args = (ids, w, sid, be, npad, bm, m.STAGE_PREP | m.STAGE_FC1 | m.STAGE_FC2, self.ws)
        if inp.dtype == "fp8":
            m.ffn_fp8(xn, inp.w1, inp.w1_scale, inp.w2, inp.w2_scale, *args, **kw)
        elif inp.dtype == "bf16":
            m.ffn_bf16(xn, inp.w1, inp.w2, *args, **kw)
        else:
            m.ffn_f32(xn, inp.w1, inp.w2, *args, **kw)
        h, y = m.ffn_intermediates(self.ws, self.T, self.E, self.H, self.I, self.k, bm, self.code)
        slots = torch.where(self.adapter < 0, -1, self.adapter * self.E + ids).int()
        plan = m.align_block(slots, self.n, bm, **kw)
        m.lora_add(y, h, self.a, self.b, *plan, bm, scale=self.scale, **kw)
        out, nxt = m.norm_out(y, w, ids, self.E, self.shared, self.gate, res, self.w_out,
                              self.w_next, 0.5, EPS, dtype=xn.dtype, **kw)
        return dict(xn=xn, res=res, logits=logits, ids=ids, w=w, out=out, next=nxt)

    def reference(self, got):
        """out and next in fp64 from the layer's own inputs; the experts are those
        the GPU's logits choose (a near tie may fall either way)."""
        inp = self.inp
        xn, s = lo.norm_in(f64(self.x), f64(self.w_in), f64(self.res), 0.75, EPS)
        logits = lo.router_logits(xn, f64(self.wr), f64(self.bias))
        ids, w = oracle.route(got["logits"].cpu().numpy(), self.k)
        assert np.array_equal(ids, got["ids"].cpu().numpy())
        size = np.abs(logits).max()
        assert np.abs(f64(got["logits"]) - logits).max() <= 2 * TOL["bf16"] * size
        T, k, I, H = self.T, self.k, self.I, self.H
        y = np.zeros((T * k, H))
        if inp.dtype == "fp8":
            dec = oracle.e4m3fn_decode
            w1 = [dec(inp.host_w1(e)) * inp.host_w1_scale()[e][:, None] for e in range(self.E)]
            w2 = [dec(inp.host_w2(e)) * inp.host_w2_scale()[e][:, None] for e in range(self.E)]
        else:
            conv = oracle.bf16_bits_to_f64 if inp.dtype == "bf16" else (lambda v: v.astype(float))
            w1 = [conv(inp.host_w1(e)) for e in range(self.E)]
            w2 = [conv(inp.host_w2(e)) for e in range(self.E)]
        adapter = self.adapter.view(-1).cpu().numpy()
        a, b, sc = f64(self.a), f64(self.b), f64(self.scale)
        for t in range(T):
            for j in range(k):
                e = ids[t, j]
                gu = w1[e] @ xn[t]
                h = gu[:I] / (1 + np.exp(-gu[:I])) * gu[I:]
                v = w2[e] @ h
                if adapter[t] >= 0:
                    q = adapter[t] * self.E + e
                    v = v + sc[q] * (b[q] @ (a[q] @ h))
                y[t * k + j] = v
        out, nxt = lo.norm_out(y, f64(got["w"]), ids, self.E, f64(self.shared), f64(self.gate), s,
                               f64(self.w_out), f64(self.w_next), 0.5, EPS)
        return dict(xn=xn, res=s, out=out, next=nxt)


@functools.lru_cache(maxsize=None)
def layer(*args):
    return Layer(*args)


LAYERS = [(5, 8, 256, 128, 2, "bf16", 16), (24, 16, 512, 256, 4, "bf16", 64),
          (40, 4, 256, 384, 2, "bf16", 256), (24, 16, 512, 256, 4, "fp8", 64),
          (40, 4, 256, 256, 2, "fp8", 256), (9, 8, 200, 136, 3, "bf16", 16),
          (6, 8, 256, 128, 2, "f32", 16)]


@pytest.mark.parametrize("T,E,H,I,k,dtype,block_m", LAYERS)
def test_layer_parity(T, E, H, I, k, dtype, block_m):
    say(f"layer T={T} E={E} H={H} I={I} k={k} {dtype} block_m={block_m}")
    L = layer(T, E, H, I, k, dtype, block_m)
    got = L.run()
    torch.cuda.synchronize()
    ref = L.reference(got)
    for name in ("xn", "res", "out", "next"):
        err = oracle.normwise_rel_err(f64(got[name]), ref[name])
        print(f"    {name}: {err:.2e}", flush=True)
        assert err <= TOL[dtype], name
    again = L.run()
    for name, t in got.items():
        assert torch.equal(t, again[name]), name


def test_layer_on_a_side_stream():
    say("layer on a side stream, another layer on the current one")
    L, other = layer(*LAYERS[1]), layer(*LAYERS[0])
    ref = {n: t.clone() for n, t in L.run().items()}
    ref_other = {n: t.clone() for n, t in other.run().items()}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):        # the elementwise step between the calls runs there too
            got = L.run(stream=s)
        here = other.run()
        torch.cuda.synchronize()
        for n in ref:
            assert torch.equal(got[n], ref[n]) and torch.equal(here[n], ref_other[n]), n


@pytest.mark.parametrize("args", [LAYERS[1], LAYERS[3]], ids=["bf16", "fp8"])
def test_layer_captured(args):
    say(f"layer captured: {args}")
    L = layer(*args)
    x0 = L.x.clone()
    x1 = rand(gen(77), *x0.shape, dtype="bf16")
    want = []
    for x in (x0, x1):
        L.x.copy_(x)
        want.append({n: t.clone() for n, t in L.run().items()})
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        L.run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = L.run()
    for i in range(5):
        L.x.copy_((x0, x1)[i % 2])
        graph.replay()
        torch.cuda.synchronize()
        for n in got:
            assert torch.equal(got[n], want[i % 2][n]), (i, n)
        (L.x.float() @ L.x.float().t()).sum()             # eager work of the program in between
        L.run()
        torch.cuda.synchronize()
    L.x.copy_(x0)


def test_two_calls_at_once():
    # the same inputs, outputs and workspaces of their own, on two streams
    say("lora_add and norm_out on two streams at once")
    m = moe()
    g = gen(9)
    S, n, r, K, N = 300, 5, 16, 512, 1024
    x, y = rand(g, S, K, dtype="bf16"), rand(g, S, N, dtype="bf16")
    a, b = rand(g, n, r, K, dtype="bf16"), rand(g, n, N, r, dtype="bf16")
    ids = torch.randint(-1, n, (S, 1), generator=g).int().cuda()
    plan = m.align_block(ids, n, 64)
    ref = m.lora_add(y, x, a, b, *plan, 64, out=y.clone())
    w = torch.rand((S // 2, 2), generator=g).cuda()
    ref_n, _ = m.norm_out(y, w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[y.clone() for _ in range(4)] for _ in streams]
    norms = [[None] * 4 for _ in streams]
    torch.cuda.synchronize()
    for i in range(4):
        for q, s in enumerate(streams):
            m.lora_add(y, x, a, b, *plan, 64, out=outs[q][i], stream=s)
            norms[q][i], _ = m.norm_out(y, w, stream=s)
    torch.cuda.synchronize()
    for q in range(2):
        for i in range(4):
            assert torch.equal(outs[q][i], ref) and torch.equal(norms[q][i], ref_n)


def test_prepared_calls():
    say("prepared calls")
    m = moe()
    g = gen(10)
    x, w = rand(g, 16, 512, dtype="bf16"), rand(g, 512)
    wr = rand(g, 32, 512, dtype="bf16")
    out, res = torch.empty_like(x), torch.empty_like(x)
    logits = torch.empty((16, 32), device="cuda")
    calls = [m.norm_in(x, w, x, out=out, residual_out=res, prepare=True),
             m.router_logits(out, wr, out=logits, prepare=True)]
    assert all(isinstance(c, m.Prepared) for c in calls)
    ref, _ = m.norm_in(x, w, x)
    ref_l = m.router_logits(ref, wr)
    for _ in range(3):
        for c in calls:
            c()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(logits, ref_l)
        out.zero_()
        logits.zero_()
