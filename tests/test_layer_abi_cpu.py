"""The operators around the FFN reject bad arguments on the host before any HIP
call, and their binding refuses what the C ABI could not see (no GPU needed)."""
import ctypes

import pytest
import torch

m = pytest.importorskip("moe_expert_ffn_router_amd")
lib = m.lib
OK, NULL, SHAPE, ALIGN, WORKSPACE, UNSUP = 0, 1, 2, 3, 4, 5
F32, BF16, FP8 = 0, 1, 2
P = 0x1000  # a fake device address: never dereferenced on these paths
INF = float("inf")


def norm_in(x=P, res=P, w=P, alpha=1.0, eps=1e-6, T=4, H=64, dt=BF16, ro=P, out=P):
    return lib.moe_norm_in(x, res, w, alpha, eps, T, H, dt, ro, out, None)


def test_norm_in_validation():
    assert norm_in(T=0, x=None, out=None) == OK
    assert norm_in(dt=FP8) == UNSUP and norm_in(dt=7) == UNSUP
    assert norm_in(T=-1) == SHAPE and norm_in(T=1 << 24) == SHAPE
    for H in (0, -8, 4, 12, 16392):
        assert norm_in(H=H) == SHAPE, H
    assert norm_in(H=12, dt=F32, x=None) == NULL           # a multiple of 4: accepted
    assert norm_in(H=6, dt=F32) == SHAPE
    assert norm_in(H=16384, x=None) == NULL                # the longest row
    for eps in (-1e-6, INF, float("nan")):
        assert norm_in(eps=eps) == UNSUP, eps
    assert norm_in(eps=0.0, x=None) == NULL
    for name in ("x", "w", "out"):
        assert norm_in(**{name: None}) == NULL, name
    for name in ("x", "res", "w", "ro", "out"):
        assert norm_in(**{name: P + 8}) == ALIGN, name
    assert norm_in(T=0, H=12) == SHAPE


def test_norm_outputs_apart():
    # 4 rows of 64 bf16: 512 bytes
    assert norm_in(ro=P, out=P) == UNSUP and norm_in(ro=P, out=P + 496) == UNSUP
    assert norm_in(ro=P + 16, out=P) == UNSUP
    Q = 1 << 30
    assert norm_out(out=Q, nxt=Q) == UNSUP and norm_out(out=Q + 496, nxt=Q) == UNSUP
    assert norm_out(out=P, nxt=Q) == UNSUP                   # y: 8 rows, 1024 bytes
    assert norm_out(out=Q, nxt=P + 1008) == UNSUP
    assert norm_out(out=P + 1008, nw=None, nxt=None) == UNSUP
    assert norm_out(out=P - 496, nw=None, nxt=None) == UNSUP


def test_outputs_are_not_part_of_an_input():
    # rows of 64 bf16, 512 bytes of them; the very buffer is allowed and tested on the GPU
    Q, R, Z = 1 << 30, 1 << 31, 1 << 32
    for d in (128, -128, 496, -496):
        assert norm_in(x=Q, res=R, ro=None, out=Q + d) == UNSUP
        assert norm_in(x=Q, res=R, ro=None, out=R + d) == UNSUP
        assert norm_in(x=Q, res=R, ro=Q + d, out=Z) == UNSUP
        assert norm_in(x=Q, res=R, ro=R + d, out=Z) == UNSUP
        assert norm_out(res=Q, shared=R, out=Q + d, nw=None, nxt=None) == UNSUP
        assert norm_out(res=Q, shared=R, out=R + d, nw=None, nxt=None) == UNSUP
        assert norm_out(res=Q, shared=R, out=Z, nxt=Q + d) == UNSUP
        assert norm_out(res=Q, shared=R, out=Z, nxt=R + d) == UNSUP
    # logits: 4 x 8 fp32, 128 bytes; x 512 bytes, w 1024
    for out in (Q, Q + 508, Q - 124, R, R + 1020, R - 124):
        assert router(x=Q, w=R, out=out) == UNSUP


def norm_out(y=P, ydt=BF16, ids=P, wts=P, shared=P, gate=P, res=P, w=P, nw=P, scale=1.0,
             eps=1e-6, T=4, E=8, H=64, k=2, dt=BF16, out=P, nxt=P):
    return lib.moe_norm_out(y, ydt, ids, wts, shared, gate, res, w, nw, scale, eps, T, E, H, k,
                            dt, out, nxt, None)


def test_norm_out_validation():
    assert norm_out(T=0, y=None, out=None) == OK
    assert norm_out(dt=FP8) == UNSUP and norm_out(ydt=FP8) == UNSUP
    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(H=12), dict(H=0), dict(H=16392),
                dict(T=1 << 22, k=4), dict(T=1 << 30, k=1 << 30)):
        assert norm_out(**bad) == SHAPE, bad
    assert norm_out(H=12, dt=F32) == SHAPE                  # y is bf16
    assert norm_out(H=12, dt=F32, ydt=F32, y=None) == NULL
    assert norm_out(E=0, ids=None, y=None) == NULL          # E is ignored without ids
    assert norm_out(E=1, k=8, y=None) == NULL               # k > E: a small shard
    for eps in (-1.0, INF, float("nan")):
        assert norm_out(eps=eps) == UNSUP
    assert norm_out(out=None) == NULL
    assert norm_out(wts=None) == NULL                       # k = 2 needs weights
    assert norm_out(shared=None) == NULL                    # a gate without shared
    assert norm_out(nw=None) == NULL and norm_out(nxt=None) == NULL
    for name in ("y", "shared", "res", "w", "nw", "out", "nxt"):
        assert norm_out(**{name: P + 8}) == ALIGN, name
    for name in ("ids", "wts", "gate"):
        assert norm_out(**{name: P + 2}) == ALIGN, name


def router(x=P, xdt=BF16, w=P, wdt=BF16, bias=P, T=4, E=8, H=64, out=P):
    return lib.moe_router_logits(x, xdt, w, wdt, bias, T, E, H, out, None)


def test_router_validation():
    assert router(T=0, x=None, out=None) == OK
    assert router(xdt=FP8) == UNSUP and router(wdt=FP8) == UNSUP
    assert router(xdt=F32, wdt=BF16) == UNSUP
    for bad in (dict(T=-1), dict(E=0), dict(E=1025), dict(H=0), dict(H=12), dict(H=4), dict(H=1 << 24),
                dict(T=1 << 24), dict(T=(1 << 31) // 8, E=8)):
        assert router(**bad) == SHAPE, bad
    for name in ("x", "w", "out"):
        assert router(**{name: None}) == NULL, name
    assert router(x=P + 8) == ALIGN and router(w=P + 8) == ALIGN
    assert router(bias=P + 2) == ALIGN and router(out=P + 1) == ALIGN


def lora(x=P, xdt=BF16, ldx=64, a=P, b=P, scale=P, sid=P, be=P, npad=P, S=4, n=3, K=64, N=128,
         r=16, M=16, ws=P, wsb=1 << 40, y=P, ydt=BF16, ldy=128, out=P, ldo=128):
    return lib.moe_lora_add(x, xdt, ldx, a, b, scale, sid, be, npad, S, n, K, N, r, M, ws, wsb, y,
                            ydt, ldy, out, ldo, None)


def test_lora_validation():
    assert lora(S=0, x=None, y=None, ws=None) == OK
    assert lora(xdt=FP8) == UNSUP and lora(ydt=FP8) == UNSUP
    for bad in (dict(S=-1), dict(S=1 << 24), dict(n=0), dict(n=1025), dict(K=0), dict(K=12),
                dict(K=1 << 24, ldx=1 << 24), dict(N=1 << 24, ldy=1 << 24, ldo=1 << 24),
                dict(N=0), dict(N=12), dict(r=0), dict(r=4), dict(r=12), dict(r=264), dict(M=0),
                dict(M=12), dict(M=512), dict(ldx=56), dict(ldx=68), dict(ldy=120), dict(ldy=132),
                dict(ldo=120), dict(ldo=132)):
        assert lora(**bad) == SHAPE, bad
    assert lora(xdt=F32, ldx=68, x=None) == NULL            # fp32 rows: a multiple of 4
    assert lora(xdt=F32, ldx=66) == SHAPE
    assert lora(ydt=F32, ldy=132, ldo=136, x=None) == NULL
    for name in ("x", "a", "b", "sid", "be", "npad", "ws", "y", "out"):
        assert lora(**{name: None}) == NULL, name
    for name in ("x", "a", "b", "y", "out"):
        assert lora(**{name: P + 8}) == ALIGN, name
    for name in ("scale", "sid", "be", "npad"):
        assert lora(**{name: P + 2}) == ALIGN, name
    assert lora(ws=P + 128) == ALIGN
    need = lib.moe_lora_workspace_bytes(4, 3, 64, 16, 16)
    assert need >= 4 * 16 * 4 and need % 256 == 0
    assert lora(wsb=need - 1) == WORKSPACE
    for bad in ((-1, 3, 64, 16, 16), (4, 0, 64, 16, 16), (4, 3, 60, 16, 16), (4, 3, 64, 12, 16),
                (4, 3, 64, 16, 3)):
        assert lib.moe_lora_workspace_bytes(*bad) == 0, bad
    # out apart from x and, unless it is y, from y: rows of 16 columns of fp32 here, 64
    # bytes each, in a matrix of 256-byte rows
    Q = 1 << 30
    apart = dict(S=4, K=16, N=16, xdt=F32, ydt=F32, ldx=64, ldy=64, ldo=64, y=Q, wsb=need * 8)

    def probe(**kw):
        return lora(**{**apart, **kw})
    for out, st in ((P, UNSUP), (P + 48, UNSUP), (P + 256 - 48, UNSUP), (P + 256 * 3, UNSUP),
                    (Q + 16, UNSUP), (Q + 256, UNSUP), (Q - 48, UNSUP)):
        assert probe(x=P, out=out) == st, hex(out)
    assert probe(x=P, out=P + 64, ldo=68) == UNSUP           # strides that cross
    assert probe(x=P, y=P + 64, out=P + 64, ldo=68, ldy=64) == UNSUP
    # the workspace never shrinks as the batch grows
    last = 0
    for S in (0, 1, 2, 17, 64, 65, 300, 4096, 100000):
        now = lib.moe_lora_workspace_bytes(S, 8, 4096, 64, 64)
        assert now >= last and now >= S * 64 * 4
        last = now


def intermediates(T, E, H, I, k, M, dt):
    h, y = ctypes.c_size_t(), ctypes.c_size_t()
    hd, yd = ctypes.c_int(), ctypes.c_int()
    st = lib.moe_ffn_intermediates(T, E, H, I, k, M, dt, ctypes.byref(h), ctypes.byref(hd),
                                   ctypes.byref(y), ctypes.byref(yd))
    return st, h.value, hd.value, y.value, yd.value


def test_ffn_intermediates():
    T, E, H, I, k = 16, 64, 4096, 1536, 8
    S = T * k
    assert intermediates(T, E, H, I, k, 64, BF16) == (OK, 0, BF16, S * I * 2, BF16)
    assert intermediates(T, E, H, I, k, 64, 3) == (OK, 0, BF16, S * I * 2, BF16)
    assert intermediates(T, E, H, I, k, 64, F32) == (OK, 0, F32, S * I * 4, F32)
    st, h, hd, y, yd = intermediates(T, E, H, I, k, 64, FP8)
    assert (st, h, hd, yd) == (OK, 0, F32, F32) and y >= S * I * 5 + S * 4 + T * H + T * 4
    # the W8A8 grouped-GEMM tiles keep bf16 in the same places; off their grid they do not run
    assert intermediates(T, E, H, I, k, 256, FP8) == (OK, 0, BF16, y, BF16)
    assert intermediates(T, E, H, I, k, 128, FP8)[2] == BF16
    assert intermediates(T, E, H + 8, I, k, 256, FP8)[2] == F32
    assert intermediates(T, E, 128, I, k, 256, FP8)[2] == F32
    assert intermediates(T, E, H, I, k, 256, 4)[2] == F32
    for args, st in (((T, E, 12, I, k, 64, BF16), SHAPE), ((T, E, H, 64, k, 64, 3), SHAPE),
                     ((T, E, H, I, 65, 64, BF16), SHAPE), ((T, E, H, I, k, 48, BF16), SHAPE),
                     ((T, E, H, I, k, 64, 9), UNSUP)):
        assert intermediates(*args)[0] == st, args
    assert lib.moe_ffn_intermediates(T, E, H, I, k, 64, BF16, None, None, None, None) == NULL
    for dt in (F32, BF16, FP8, 3, 4):                      # y fits behind its offset
        _, _, _, y, yd = intermediates(T, E, H, I, k, 64, dt)
        assert y + S * H * (2 if yd == BF16 else 4) <= lib.moe_ffn_workspace_bytes(T, E, H, I, k,
                                                                                   64, dt)


def test_binding_refuses_host_tensors_and_wrong_types():
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros(64)
    with pytest.raises(ValueError, match="device"):
        m.norm_in(x, w)
    with pytest.raises(ValueError, match="device"):
        m.norm_out(x)
    with pytest.raises(ValueError, match="device"):
        m.router_logits(x, torch.zeros((8, 64), dtype=torch.bfloat16))
    a, b = (torch.zeros((3, 8, 64), dtype=torch.bfloat16),
            torch.zeros((3, 64, 8), dtype=torch.bfloat16))
    i = torch.zeros(256, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        m.lora_add(x, x, a, b, i, i, i, 16)
    with pytest.raises(TypeError):
        m.norm_in(x.half(), w)
    with pytest.raises(TypeError):
        m.norm_out([1.0])
    with pytest.raises(TypeError):
        m.router_logits(x, x.to(torch.float16))
    with pytest.raises(ValueError, match="dimensions"):
        m.norm_in(x[0], w)
    with pytest.raises(ValueError, match="dimensions"):
        m.lora_add(x, x, a[0], b, i, i, i, 16)
    with pytest.raises(ValueError, match="device"):
        m.ffn_intermediates(torch.zeros(1 << 20, dtype=torch.uint8), 4, 8, 128, 128, 2, 16, 1)
    with pytest.raises(m.MoEError):
        m.ffn_intermediates(torch.zeros(16, dtype=torch.uint8), 4, 8, 100, 128, 2, 16, 1)
