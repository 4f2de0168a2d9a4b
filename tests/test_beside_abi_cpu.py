"""The operators beside the FFN reject bad arguments on the host before any HIP call, and their
binding refuses what the C ABI could not see (no GPU needed; the addresses are never read)."""
import pytest
import torch

m = pytest.importorskip("moe_expert_ffn_router_amd")
lib = m.lib
OK, NULL, SHAPE, ALIGN, WORKSPACE, UNSUP = 0, 1, 2, 3, 4, 5
F32, BF16, FP8 = 0, 1, 2
INF, NAN = float("inf"), float("nan")
# operands of a call, 4 GiB apart
A, B, C, D, E_, F, G, H_, J, K_, L = ((i + 1) << 32 for i in range(11))


def touching(at, operand_bytes, out_bytes):
    """Addresses for an output of out_bytes that shares 16 bytes or more with the operand."""
    return {at, at + operand_bytes - 16, at - out_bytes + 16}


# ------------------------------------------------- rows in expert order ---

def dispatch(x=A, ids=B, sid=C, npad=D, T=16, E=8, H=64, k=2, R=48, dt=BF16, rows=E_, at=F):
    return lib.moe_dispatch(x, ids, sid, npad, T, E, H, k, R, dt, rows, at, None)


def combine(rows=A, rdt=BF16, at=B, wts=C, T=16, H=64, k=2, R=48, dt=BF16, out=D):
    return lib.moe_combine(rows, rdt, at, wts, T, H, k, R, dt, out, None)


def dispatch_bwd(rows=A, at=B, T=16, H=64, k=2, R=48, dt=BF16, dx=D):
    return lib.moe_dispatch_backward(rows, at, T, H, k, R, dt, dx, None)


def combine_bwd(dout=A, dt=BF16, rows=B, rdt=BF16, at=C, wts=D, sid=E_, npad=F, T=16, H=64, k=2,
                R=48, drows=G, dw=H_):
    return lib.moe_combine_backward(dout, dt, rows, rdt, at, wts, sid, npad, T, H, k, R, drows, dw,
                                    None)


CALLS = [dispatch, combine, dispatch_bwd, combine_bwd]


@pytest.mark.parametrize("call", CALLS)
def test_rows_sizes(call):
    assert call(T=0, R=0) == OK and call(T=0, at=None) == OK
    for bad in (dict(T=-1), dict(k=0), dict(H=0), dict(H=-8), dict(H=(1 << 20) + 1), dict(R=0),
                dict(R=-1), dict(R=1 << 25), dict(T=1 << 23, k=2), dict(T=1 << 30, k=1 << 30),
                dict(T=1 << 22, H=1 << 15, k=1), dict(R=1 << 22, H=1 << 15)):
        assert call(**bad) == SHAPE, bad
    assert call(dt=FP8) == UNSUP and call(dt=7) == UNSUP
    assert call(at=None) == NULL and call(k=64, at=None) == NULL   # k may exceed E
    assert call(at=B + 2) == ALIGN
    for H in (1, 3, 1031):                                        # any length
        assert call(H=H, at=None) == NULL


def test_dispatch_validation():
    assert dispatch(E=0) == SHAPE and dispatch(E=-1) == SHAPE
    for name in ("x", "ids", "sid", "npad", "rows", "at"):
        assert dispatch(**{name: None}) == NULL, name
    for name in ("ids", "sid", "npad", "at"):
        assert dispatch(**{name: A + 2}) == ALIGN, name
    for name in ("x", "rows"):
        assert dispatch(**{name: L + 1}) == ALIGN and dispatch(dt=F32, **{name: L + 2}) == ALIGN


def test_combine_validation():
    assert combine(rdt=FP8) == UNSUP
    for name in ("rows", "out", "at"):
        assert combine(**{name: None}) == NULL, name
    assert combine(wts=C + 2) == ALIGN and combine(out=D + 1) == ALIGN
    assert combine(rdt=F32, rows=A + 2) == ALIGN and dispatch_bwd(dx=D + 1) == ALIGN
    assert dispatch_bwd(rows=None) == NULL and dispatch_bwd(dx=None) == NULL


def test_combine_backward_validation():
    assert combine_bwd(rdt=FP8) == UNSUP
    for name in ("dout", "rows", "at", "sid", "npad", "drows"):
        assert combine_bwd(**{name: None}) == NULL, name
    for name in ("wts", "sid", "npad", "dw"):
        assert combine_bwd(**{name: L + 2}) == ALIGN, name
    for name in ("dout", "rows", "drows"):
        assert combine_bwd(**{name: L + 1}) == ALIGN, name


def test_rows_outputs_apart():
    # x 16 x 64 bf16: 2048 bytes; rows 48 x 64: 6144; slots 128; sorted_ids 192
    for at, size in ((A, 2048), (B, 128), (C, 192), (D, 16)):
        for out in touching(at, size, 6144):
            assert dispatch(rows=out) == UNSUP
        for out in touching(at, size, 128):
            assert dispatch(at=out) == UNSUP
    for out in touching(F, 128, 6144):
        assert dispatch(rows=out) == UNSUP
    for at, size in ((A, 6144), (B, 128), (C, 128)):
        for out in touching(at, size, 2048):
            assert combine(out=out) == UNSUP
            if at != C:
                assert dispatch_bwd(dx=out) == UNSUP
    for at, size in ((A, 2048), (C, 128), (D, 128), (E_, 192), (F, 16)):
        for out in touching(at, size, 6144):
            assert combine_bwd(drows=out) == UNSUP
        for out in touching(at, size, 128):
            assert combine_bwd(dw=out) == UNSUP
    for out in touching(G, 6144, 128):
        assert combine_bwd(dw=out) == UNSUP
    for out in touching(B, 6144, 128):
        assert combine_bwd(dw=out) == UNSUP
    for d in (128, -128, 6128, -6128):                       # the very buffer is fine
        assert combine_bwd(drows=B + d) == UNSUP


# ------------------------------------------------------------ layer norm ---

def norm(x=A, res=B, w=C, b=D, alpha=1.0, eps=1e-5, T=4, H=64, dt=BF16, ro=E_, out=F):
    return lib.moe_layer_norm(x, res, w, b, alpha, eps, T, H, dt, ro, out, None)


def norm_bwd(dout=A, s=B, w=C, dro=D, alpha=1.0, eps=1e-5, T=4, H=64, dt=BF16, dx=E_, dr=F, dw=G,
             db=H_, ws=J, wsb=1 << 30):
    return lib.moe_layer_norm_backward(dout, s, w, dro, alpha, eps, T, H, dt, dx, dr, dw, db, ws,
                                       wsb, None)


@pytest.mark.parametrize("call", [norm, norm_bwd])
def test_layer_norm_sizes(call):
    for bad in (dict(T=-1), dict(T=1 << 24), dict(H=0), dict(H=-1), dict(H=16385)):
        assert call(**bad) == SHAPE, bad
    for eps in (-1e-6, INF, NAN):
        assert call(eps=eps) == UNSUP, eps
    assert call(dt=FP8) == UNSUP and call(dt=9) == UNSUP


def test_layer_norm_validation():
    assert norm(T=0, x=None, out=None) == OK
    assert norm(x=None) == NULL and norm(out=None) == NULL and norm(x=None, H=1031) == NULL
    for name in ("x", "res", "ro", "out"):
        assert norm(**{name: L + 1}) == ALIGN and norm(dt=F32, **{name: L + 2}) == ALIGN, name
    assert norm(w=C + 2) == ALIGN and norm(b=D + 1) == ALIGN
    # rows of 64 bf16: 512 bytes
    assert norm(ro=F) == UNSUP and norm(ro=F + 496) == UNSUP
    for d in (128, -128, 496, -496):
        for at in (A, B):
            assert norm(out=at + d) == UNSUP and norm(ro=at + d) == UNSUP
    for at in (C, D):
        for out in touching(at, 256, 512):
            assert norm(out=out) == UNSUP and norm(ro=out) == UNSUP


def test_layer_norm_backward_validation():
    used = lib.moe_layer_norm_backward_workspace_bytes(4, 64)
    assert used >= 2 * 64 * 4 and lib.moe_layer_norm_backward_workspace_bytes(0, 64) == 0
    assert lib.moe_layer_norm_backward_workspace_bytes(-1, 64) == 0
    assert lib.moe_layer_norm_backward_workspace_bytes(4, 20000) == 0
    sizes = [lib.moe_layer_norm_backward_workspace_bytes(T, 640) for T in range(0, 20000, 7)]
    assert sizes == sorted(sizes)                            # holds for every smaller T
    for name in ("dout", "s", "dx", "ws"):
        assert norm_bwd(**{name: None}) == NULL, name
    assert norm_bwd(ws=None, dw=None, dout=None) == NULL
    assert norm_bwd(wsb=used - 1) == WORKSPACE
    assert norm_bwd(wsb=0, dw=None) == WORKSPACE             # dbias needs it too
    for name in ("dout", "s", "dro", "dx", "dr"):
        assert norm_bwd(**{name: L + 1}) == ALIGN, name
    for name in ("w", "dw", "db"):
        assert norm_bwd(**{name: L + 2}) == ALIGN, name
    assert norm_bwd(ws=J + 8) == ALIGN


def test_layer_norm_backward_outputs_apart():
    used = lib.moe_layer_norm_backward_workspace_bytes(4, 64)
    assert norm_bwd(dr=E_) == UNSUP and norm_bwd(dr=E_ + 496) == UNSUP
    for d in (128, -128, 496, -496):
        for at in (A, B, D):
            assert norm_bwd(dx=at + d) == UNSUP and norm_bwd(dr=at + d) == UNSUP
    for out in touching(C, 256, 512):
        assert norm_bwd(dx=out) == UNSUP and norm_bwd(dr=out) == UNSUP
    for at, size in ((A, 512), (B, 512), (C, 256), (D, 512), (E_, 512), (F, 512)):
        for out in touching(at, size, 256):
            assert norm_bwd(dw=out) == UNSUP and norm_bwd(db=out) == UNSUP
        for ws in touching(at, size, used):
            assert norm_bwd(ws=ws) == UNSUP
    for out in touching(G, 256, 256):
        assert norm_bwd(db=out) == UNSUP
    for at in (G, H_):
        for ws in touching(at, 256, used):
            assert norm_bwd(ws=ws) == UNSUP


# ---------------------------------------------------------------- linear ---

def linear(x=A, ldx=64, w=B, bias=C, act=0, gated=0, res=D, ldr=32, T=4, N=32, K=64, dt=BF16,
           odt=BF16, ws=J, wsb=1 << 30, out=E_, ldo=32):
    return lib.moe_linear(x, ldx, w, bias, act, gated, res, ldr, T, N, K, dt, odt, ws, wsb, out,
                          ldo, None)


def test_linear_validation():
    assert linear(T=0, x=None, out=None) == OK
    assert linear(dt=FP8) == UNSUP and linear(odt=FP8) == UNSUP
    assert linear(act=-1) == UNSUP and linear(act=5) == UNSUP
    for bad in (dict(T=-1), dict(T=1 << 24), dict(N=0), dict(N=1 << 24), dict(K=0), dict(K=4),
                dict(K=60), dict(T=1 << 20, N=1 << 17, ldo=1 << 17, ldr=1 << 17),
                dict(K=1 << 21, ldx=1 << 21), dict(ldx=56), dict(ldx=68),
                dict(ldx=1 << 21), dict(ldo=31), dict(ldr=31), dict(ldo=1 << 31),
                dict(ldr=1 << 31), dict(ldx=66, dt=F32)):
        assert linear(**bad) == SHAPE, bad
    # gated: the rows of w count
    assert linear(gated=1, N=1 << 23, ldo=1 << 23, ldr=1 << 23) == SHAPE
    assert linear(gated=1, N=(1 << 23) - 1, ldo=1 << 23, ldr=1 << 23, x=None) == NULL
    assert linear(ldx=68, dt=F32, x=None) == NULL
    assert linear(res=None, ldr=0, x=None) == NULL            # ldr is ignored
    for name in ("x", "w", "out"):
        assert linear(**{name: None}) == NULL, name
    assert linear(x=A + 8) == ALIGN and linear(w=B + 8) == ALIGN and linear(bias=C + 2) == ALIGN
    assert linear(out=E_ + 1) == ALIGN and linear(odt=F32, out=E_ + 2) == ALIGN
    assert linear(res=D + 1) == ALIGN
    assert lib.moe_linear_workspace_bytes(4, 32, 60, 0, BF16) == 0
    assert lib.moe_linear_workspace_bytes(4, 32, 64, 0, FP8) == 0


@pytest.mark.parametrize("T,N,K,gated,dt", [(64, 64, 8192, 0, BF16), (300, 520, 4096, 1, BF16),
                                            (64, 64, 4096, 0, F32), (1, 64, 16384, 1, F32)])
def test_linear_workspace(T, N, K, gated, dt):
    used = lib.moe_linear_workspace_bytes(T, N, K, gated, dt)
    size = 2 if dt == BF16 else 4
    call = dict(T=T, N=N, K=K, gated=gated, dt=dt, odt=dt, ldx=K, ldo=N, ldr=N, wsb=used)
    if not used:
        return
    assert linear(ws=None, **call) == NULL and linear(ws=J + 128, **call) == ALIGN
    assert linear(**{**call, "wsb": used - 1}) == WORKSPACE
    n = N * (2 if gated else 1)
    for at, bytes_ in ((A, T * K * size), (B, n * K * size), (C, n * 4), (D, T * N * size),
                       (E_, T * N * size)):
        for ws in (at, at - used + 256, at + (bytes_ - 1) // 256 * 256):
            assert linear(ws=ws, **call) == UNSUP, hex(at)


def test_linear_outputs_apart():
    # x 4 x 64 bf16: 512 bytes, w 32 x 64: 4096, bias 128, out 256
    for at, size in ((A, 512), (B, 4096), (C, 128)):
        for out in touching(at, size, 256):
            assert linear(out=out) == UNSUP
    for out in (D + 16, D - 16, D + 240, D - 240):           # a part of residual
        assert linear(out=out) == UNSUP
    assert linear(out=D, ldo=40) == UNSUP                    # residual with another stride
    assert linear(out=B + 4096 - 64, gated=1) == UNSUP and linear(out=B + 8192 - 64, gated=1) == UNSUP
    # the last row of a strided output in w
    assert linear(out=B - 3 * 4096, ldo=2048) == UNSUP


# --------------------------------------------------------------- binding ---

def test_host_tensors_are_refused():
    x, ids = torch.zeros((4, 64)), torch.zeros((4, 2), dtype=torch.int32)
    sid, n = torch.zeros(8, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    w = torch.zeros((8, 64))
    for call in (lambda: m.dispatch(x, ids, 4, sid, n), lambda: m.dispatch_backward(x, ids),
                 lambda: m.combine(x, ids), lambda: m.layer_norm(x),
                 lambda: m.combine_backward(x, x, ids, None, sid, n),
                 lambda: m.layer_norm_backward(x, x), lambda: m.linear(x, w)):
        with pytest.raises(ValueError, match="device"):
            call()


def test_wrong_types_and_ranks_are_refused():
    x = torch.zeros((4, 64))
    with pytest.raises(ValueError, match="dimensions"):
        m.linear(torch.zeros(64), x)
    with pytest.raises(ValueError, match="dimensions"):
        m.layer_norm(torch.zeros((2, 4, 64)))
    with pytest.raises(TypeError, match="dtype"):
        m.combine(x.half(), None)
    with pytest.raises(TypeError, match="Tensor"):
        m.dispatch([[0.0]], None, 4, None, None)
    with pytest.raises(TypeError, match="dtype"):
        m.layer_norm_backward(x.double(), x)


def test_linear_gated_fp32_grid():
    """Products whose tiles would be 2^23 workgroups of 512 threads, 2^32 in one dimension."""
    big = dict(gated=1, odt=BF16, res=None, x=None)
    for T, N in ((16384, (1 << 23) - 1), ((1 << 24) - 1, 8129), (16129, (1 << 23) - 1)):
        call = dict(T=T, N=N, ldo=N, **big)
        assert linear(dt=F32, **call) == SHAPE, (T, N)
        assert linear(dt=BF16, **call) == NULL and linear(dt=F32, **{**call, "gated": 0}) == NULL
        assert lib.moe_linear_workspace_bytes(T, N, 64, 1, F32) == 0
    for T, N in ((16128, (1 << 23) - 1), ((1 << 24) - 1, 8128)):
        assert linear(dt=F32, T=T, N=N, ldo=N, **big) == NULL, (T, N)
