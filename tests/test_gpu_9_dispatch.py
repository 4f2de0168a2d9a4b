"""GPU parity of the rows in expert order and back against the fp64 oracle: copies bit for bit,
sums within half a step of their type plus the fp32 arithmetic's own error."""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as lo
from tests.gpu_util import moe, say
from tests.layer_util import DT, U, close, f64, gen, rand, sentinel

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


class Routed:
    """T tokens with k slots over E experts, of which `local` are here, and their lists; a few
    tokens all of whose slots are elsewhere where local < E."""

    def __init__(self, T, k, E, local, block_m, seed, wide=0):
        g = gen(seed)
        ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
        if local < E:
            ids[::5] = torch.randint(local, E, (len(ids[::5]), k), generator=g)
            ids[1::7, 0] = -1
        self.ids = ids.int().cuda()
        self.T, self.k, self.E, self.S = T, k, local, T * k
        self.sid, _, self.npad = moe().align_block(self.ids, max(local, k), block_m)
        if local < k:      # a small shard: its lists are those without the others' slots
            mine = torch.where(self.ids < local, self.ids, -1)
            self.sid, _, self.npad = moe().align_block(mine, k, block_m)
        if wide:           # more room than the alignment needs
            self.sid = torch.cat([self.sid, torch.full((wide,), self.S, dtype=torch.int32,
                                                       device="cuda")])
        self.R, self.n = self.sid.numel(), int(self.npad)
        self.sid_h = self.sid.cpu().numpy()
        self.at = lo.places(self.sid_h, self.n, self.S).reshape(T, k)
        self.slot_rows = torch.from_numpy(self.at).int().cuda()
        self.w = torch.rand((T, k), generator=g).cuda()
        self.g = g


# T, k, E, local, block_m, H, dtype: one token to many, padded and unpadded runs, shards, rows off
# the 16-byte grid, rows longer than a wave's piece, more than 64 slots a token
CASES = [(1, 1, 1, 1, 1, 8, "bf16"), (1, 8, 64, 64, 16, 4096, "bf16"), (3, 2, 4, 4, 16, 1, "bf16"),
         (7, 3, 8, 2, 4, 24, "bf16"), (16, 8, 64, 16, 64, 1031, "bf16"),
         (33, 6, 60, 60, 1, 2056, "bf16"), (65, 4, 8, 8, 128, 520, "bf16"),
         (5, 70, 90, 45, 2, 72, "bf16"), (200, 8, 128, 128, 16, 256, "bf16"),
         (1, 2, 8, 8, 1, 4, "f32"), (9, 4, 16, 16, 8, 1030, "f32"), (31, 3, 8, 4, 32, 37, "f32"),
         (64, 8, 32, 8, 1, 4100, "f32"), (2, 64, 64, 64, 1, 12, "f32"),
         (11, 65, 80, 80, 4, 8, "f32"), (4, 8, 16, 3, 256, 8200, "bf16")]


@pytest.mark.parametrize("T,k,E,local,block_m,H,dtype", CASES)
def test_dispatch(T, k, E, local, block_m, H, dtype):
    say(f"dispatch T={T} k={k} E={E}/{local} block_m={block_m} H={H} {dtype}")
    r = Routed(T, k, E, local, block_m, T + k, wide=T % 3)
    # any bits at all: infinities, NaN with payloads, subnormal values
    x = torch.randint(-2 ** 31, 2 ** 31 - 1, (T, H), generator=r.g).int().cuda()
    x = (x >> 16).short().view(torch.bfloat16) if dtype == "bf16" else x.view(torch.float32)
    out, ok = sentinel((r.R, H), dtype)
    rows, at = moe().dispatch(x, r.ids, r.E, r.sid, r.npad, out=out)
    torch.cuda.synchronize()
    ok()
    assert np.array_equal(at.cpu().numpy(), r.at)
    ref = lo.dispatch(bits(x).cpu().numpy(), r.sid_h, r.n, k)
    assert np.array_equal(bits(rows[:r.n]).cpu().numpy(), ref)
    assert bool((rows[r.n:] == 12345.0).all()), "rows behind the last run were written"
    a, b = moe().dispatch(x, r.ids, r.E, r.sid, r.npad)      # the outputs it allocates itself
    assert torch.equal(bits(a[:r.n]), bits(rows[:r.n])) and torch.equal(b, at)


def poisoned(r, H, dtype):
    """Rows in expert order; those of no slot are NaN: nothing may read them."""
    rows = rand(r.g, r.R, H, dtype=dtype)
    none = torch.ones(r.R, dtype=torch.bool)
    none[torch.from_numpy(r.at[r.at >= 0].reshape(-1))] = False
    rows[none.cuda()] = float("nan")
    return rows


@pytest.mark.parametrize("T,k,E,local,block_m,H,dtype", CASES)
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
def test_combine(T, k, E, local, block_m, H, dtype, out_dtype):
    say(f"combine T={T} k={k} E={E}/{local} block_m={block_m} H={H} {dtype} -> {out_dtype}")
    r = Routed(T, k, E, local, block_m, 3 * T + k)
    rows = poisoned(r, H, dtype)
    w = r.w.clone()
    w[torch.from_numpy(r.at < 0).cuda()] = float("inf")      # weights of absent slots do not count
    out, ok = sentinel((T, H), out_dtype)
    moe().combine(rows, r.slot_rows, w, out=out)
    torch.cuda.synchronize()
    ok()
    # k products and sums, each off by u at most
    y, wh = np.nan_to_num(f64(rows)), f64(r.w)
    mag = lo.combine(np.abs(y), r.at, wh)
    close(out, lo.combine(y, r.at, wh), (2 * k + 1) * U * mag, out_dtype, "out")
    none = torch.from_numpy((r.at < 0).all(1)).cuda()
    assert bool((out[none] == 0).all())
    plain = moe().combine(rows, r.slot_rows, dtype=DT[out_dtype])
    close(plain, lo.combine(y, r.at), (k + 1) * U * lo.combine(np.abs(y), r.at), out_dtype, "sum")


@pytest.mark.parametrize("T,k,E,local,block_m,H,dtype", CASES)
def test_dispatch_backward(T, k, E, local, block_m, H, dtype):
    say(f"dispatch_backward T={T} k={k} E={E}/{local} block_m={block_m} H={H} {dtype}")
    r = Routed(T, k, E, local, block_m, 5 * T + k)
    drows = poisoned(r, H, dtype)
    dx, ok = sentinel((T, H), dtype)
    moe().dispatch_backward(drows, r.slot_rows, out=dx)
    torch.cuda.synchronize()
    ok()
    y = np.nan_to_num(f64(drows))
    close(dx, lo.combine(y, r.at), (k + 1) * U * lo.combine(np.abs(y), r.at), dtype, "dx")


@pytest.mark.parametrize("T,k,E,local,block_m,H,dtype", CASES)
@pytest.mark.parametrize("tok_dtype", ["bf16", "f32"])
def test_combine_backward(T, k, E, local, block_m, H, dtype, tok_dtype):
    say(f"combine_backward T={T} k={k} E={E}/{local} block_m={block_m} H={H} {tok_dtype} {dtype}")
    r = Routed(T, k, E, local, block_m, 7 * T + k, wide=T % 4)
    rows, dout = poisoned(r, H, dtype), rand(r.g, T, H, dtype=tok_dtype)
    drows, ok = sentinel((r.R, H), dtype)
    dw, ok2 = sentinel((T, k), "f32")
    moe().combine_backward(dout, rows, r.slot_rows, r.w, r.sid, r.npad, drows=drows, dweights=dw)
    torch.cuda.synchronize()
    ok()
    ok2()
    y, d = np.nan_to_num(f64(rows)), f64(dout)
    ref, ref_w = lo.combine_backward(d, y, r.at, f64(r.w), r.n)
    close(drows[:r.n], ref, U * np.abs(ref), dtype, "drows")
    assert bool((drows[r.n:] == 12345.0).all()), "rows behind the last run were written"
    _, mag = lo.combine_backward(np.abs(d), np.abs(y), r.at, f64(r.w), r.n)
    close(dw, ref_w, (H + 2) * U * mag, "f32", "dweights")
    # in place, and without weights
    again = rows.clone()
    moe().combine_backward(dout, again, r.slot_rows, r.w, r.sid, r.npad, drows=again)
    assert torch.equal(again[:r.n], drows[:r.n])
    assert torch.equal(bits(again[r.n:]), bits(rows[r.n:]))
    one, dw1 = moe().combine_backward(dout, rows, r.slot_rows, None, r.sid, r.npad)
    ref, _ = lo.combine_backward(d, y, r.at, None, r.n)
    close(one[:r.n], ref, 0.0, dtype, "drows without weights")
    assert torch.equal(dw1, dw)


def test_no_dweights():
    """The C ABI without dweights: rows are not asked for and the gradient is the same."""
    r = Routed(12, 2, 8, 4, 8, 1)
    dout = rand(r.g, 12, 264, dtype="bf16")
    m, drows = moe(), torch.zeros((r.R, 264), dtype=torch.bfloat16, device="cuda")
    s = m.lib.moe_combine_backward(dout.data_ptr(), m.MOE_DTYPE_BF16, None, m.MOE_DTYPE_BF16,
                                   r.slot_rows.data_ptr(), r.w.data_ptr(), r.sid.data_ptr(),
                                   r.npad.data_ptr(), 12, 264, 2, r.R, drows.data_ptr(), None,
                                   torch.cuda.current_stream().cuda_stream)
    assert s == m.MOE_OK
    ref, _ = m.combine_backward(dout, torch.zeros_like(drows), r.slot_rows, r.w, r.sid, r.npad)
    assert torch.equal(drows[:r.n], ref[:r.n])


def test_adjoints():
    """<dispatch(x), r> = <x, dispatch_backward(r)> and the same of combine, exactly: small whole
    numbers."""
    say("dispatch and combine against their gradients")
    r = Routed(37, 4, 16, 12, 8, 9)
    H = 264

    def whole(*shape):
        return torch.randint(-4, 5, shape, generator=r.g).float().cuda()

    x, rows, dout = whole(37, H), whole(r.R, H), whole(37, H)
    got, _ = moe().dispatch(x, r.ids, r.E, r.sid, r.npad)
    dx = moe().dispatch_backward(rows, r.slot_rows)
    assert torch.equal((got[:r.n].double() * rows[:r.n].double()).sum(),
                       (x.double() * dx.double()).sum())
    w = whole(37, 4)
    out = moe().combine(rows, r.slot_rows, w)
    drows, dw = moe().combine_backward(dout, rows, r.slot_rows, w, r.sid, r.npad)
    here = r.slot_rows >= 0
    loss = (out.double() * dout.double()).sum()
    assert torch.equal((drows[:r.n].double() * rows[:r.n].double()).sum(), loss)
    assert torch.equal((dw.double() * w.double())[here].sum(), loss)


def test_special_values_stay_in_their_rows():
    say("rows: infinities and NaN")
    r = Routed(6, 2, 4, 4, 2, 11)
    rows = rand(r.g, r.R, 72, dtype="bf16")
    bad = int(r.at[3, 1])
    rows[bad, 5] = float("inf")
    rows[bad, 6] = float("nan")
    out = moe().combine(rows, r.slot_rows, r.w)
    fine = torch.isfinite(out)
    assert bool(torch.isinf(out[3, 5])) and bool(torch.isnan(out[3, 6]))
    assert int((~fine).sum()) == 2
    dout = rand(r.g, 6, 72, dtype="bf16")
    drows, dw = moe().combine_backward(dout, rows, r.slot_rows, r.w, r.sid, r.npad)
    assert bool(torch.isfinite(drows[:r.n]).all()) and int((~torch.isfinite(dw)).sum()) == 1


def test_all_slots_elsewhere():
    say("rows: no slot here")
    m = moe()
    ids = torch.full((5, 3), 9, dtype=torch.int32, device="cuda")
    sid, _, npad = m.align_block(ids, 4, 16)
    x = torch.ones((5, 24), device="cuda")
    out, ok = sentinel((sid.numel(), 24), "f32")
    rows, at = m.dispatch(x, ids, 4, sid, npad, out=out)
    assert bool((at == -1).all()) and bool((rows == 12345.0).all())
    ok()
    assert bool((m.combine(rows, at, torch.ones((5, 3), device="cuda")) == 0).all())
    assert bool((m.dispatch_backward(rows, at) == 0).all())
    drows, dw = m.combine_backward(x, rows, at, None, sid, npad, drows=rows)
    assert bool((drows == 12345.0).all()) and bool((dw == 0).all())


def test_no_tokens():
    m = moe()
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    sid, _, npad = m.align_block(ids, 4, 16)
    rows, at = m.dispatch(torch.empty((0, 24), device="cuda"), ids, 4, sid, npad)
    assert rows.shape == (0, 24) and at.shape == (0, 2)
    assert m.combine(rows, at).shape == (0, 24)


# rows of 60 to 170 MB: both sides of the rules on what all rows together hold, and such rows off
# the 16-byte grid
LARGE = [(2000, 8, 64, 64, 16, 1880, "bf16"), (2100, 8, 64, 64, 16, 2000, "bf16"),
         (2100, 8, 64, 16, 64, 2000, "bf16"), (4200, 8, 128, 128, 1, 2000, "bf16"),
         (4200, 8, 128, 100, 128, 2001, "bf16"), (2100, 4, 8, 8, 128, 2004, "f32"),
         (4300, 4, 8, 8, 1, 2004, "f32"), (4300, 4, 8, 6, 16, 2003, "f32"),
         (300, 66, 80, 80, 1, 4096, "bf16")]


@pytest.mark.parametrize("T,k,E,local,block_m,H,dtype", LARGE)
def test_large(T, k, E, local, block_m, H, dtype):
    """Against torch on the GPU: the copies and places bit for bit, the sums in 64 bits."""
    say(f"rows T={T} k={k} E={E}/{local} block_m={block_m} H={H} {dtype}")
    r, m = Routed(T, k, E, local, block_m, 3), moe()
    x = torch.randn((T, H), generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(
        DT[dtype])
    out, ok = sentinel((r.R, H), dtype)
    rows, at = m.dispatch(x, r.ids, r.E, r.sid, r.npad, out=out)
    ok()
    assert torch.equal(at, r.slot_rows)
    slot = r.sid[:r.n].long()
    ref = x[slot.clamp(max=r.S - 1) // k]
    ref[slot >= r.S] = 0
    assert torch.equal(rows[:r.n], ref) and bool((rows[r.n:] == 12345.0).all())
    del ref
    here, place = (at >= 0), at.long().clamp(min=0)
    w = torch.where(here, r.w, 0.0)

    def total(weights, src):
        v = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(v)
        for j in range(k):
            term = src[place[:, j]].double() * weights[:, j, None].double()
            v += term
            mag += term.abs()
        return v.cpu().numpy(), mag.cpu().numpy()

    v, mag = total(w, rows)
    close(m.combine(rows, at, r.w), v, (2 * k + 1) * U * mag, dtype, "out")
    v, mag = total(here.float(), rows)
    close(m.dispatch_backward(rows, at), v, (k + 1) * U * mag, dtype, "dx")
    drows, ok = sentinel((r.R, H), dtype)
    _, dw = m.combine_backward(x, rows, at, r.w, r.sid, r.npad, drows=drows)
    ok()
    live = slot < r.S
    wt = torch.where(live, r.w.view(-1)[slot.clamp(max=r.S - 1)], 0.0)
    ref = (x[slot.clamp(max=r.S - 1) // k].float() * wt[:, None]).to(DT[dtype])
    assert torch.equal(drows[:r.n].float() + 0.0, ref.float() + 0.0)
    assert bool((drows[r.n:] == 12345.0).all())
    dots = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    mags = torch.zeros_like(dots)
    for j in range(k):
        term = x.double() * rows[place[:, j]].double() * here[:, j, None]
        dots[:, j], mags[:, j] = term.sum(1), term.abs().sum(1)
    close(dw, dots.cpu().numpy(), (H + 2) * U * mags.cpu().numpy(), "f32", "dweights")


@pytest.mark.parametrize("H,dtype", [(1 << 20, "bf16"), ((1 << 20) - 1, "bf16"), (1 << 20, "f32")])
def test_longest_rows(H, dtype):
    say(f"rows of {H} {dtype}")
    r, m = Routed(3, 2, 4, 3, 2, 5), moe()
    x = rand(r.g, 3, H, dtype=dtype)
    rows, at = m.dispatch(x, r.ids, r.E, r.sid, r.npad)
    assert torch.equal(bits(rows[:r.n]).cpu(), torch.from_numpy(
        lo.dispatch(bits(x).cpu().numpy(), r.sid_h, r.n, 2)))
    y = f64(rows[:r.n])
    close(m.combine(rows, at, r.w), lo.combine(y, r.at, f64(r.w)),
          5 * U * lo.combine(np.abs(y), r.at, f64(r.w)), dtype, "out")
    drows, dw = m.combine_backward(x, rows, at, r.w, r.sid, r.npad)
    ref, ref_w = lo.combine_backward(f64(x), y, r.at, f64(r.w), r.n)
    _, mag = lo.combine_backward(np.abs(f64(x)), np.abs(y), r.at, f64(r.w), r.n)
    close(drows[:r.n], ref, U * np.abs(ref), dtype, "drows")
    close(dw, ref_w, (H / 64 + 8) * U * mag, "f32", "dweights")   # a lane adds H / 64, then six steps


def test_offsets_past_32_bits():
    """2^21 + 3 slots of rows of 2056 bf16: more than 2^32 elements; the last rows are checked."""
    T, k, H = (1 << 21) + 3, 1, 2056
    say(f"rows: {T} x {H} bf16")
    m = moe()
    # two experts, so that the last tokens lie in the middle and at the end
    ids = (torch.arange(T, device="cuda") % 2).int().view(T, 1)
    sid, _, npad = m.align_block(ids, 2, 1)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x[-4:] = rand(gen(1), 4, H, dtype="bf16")
    rows, at = m.dispatch(x, ids, 2, sid, npad)
    assert torch.equal(rows[at[-4:, 0].long()], x[-4:])
    del x
    w = torch.full((T, 1), 0.5, device="cuda")
    out = m.combine(rows, at, w)
    assert torch.equal(out[-4:].float(), rows[at[-4:, 0].long()].float() * 0.5)
    drows, dw = m.combine_backward(out, rows, at, w, sid, npad, drows=rows)
    assert torch.equal(drows[at[-4:, 0].long()].float(), out[-4:].float() * 0.5)


# T, k, H, dtype: rows of 64 MB and more whose last words are fewer than a wave's lanes, and than a
# token's slots: 513 and 1025 words of 16 bytes (on and off their grid; together on both sides of
# 128 MB), rows of fewer words than slots, rows below 16 bytes (words of an element)
TAILS = [(1100, 8, 4104, "bf16"), (2200, 8, 4104, "bf16"), (1100, 8, 4100, "bf16"),
         (2200, 8, 4100, "bf16"), (1100, 8, 2052, "f32"), (2200, 8, 2049, "f32"),
         (560, 8, 8200, "bf16"), (140, 66, 4104, "bf16"), (270, 66, 4098, "bf16"),
         (1700, 66, 320, "bf16"), (3400, 66, 319, "bf16"), (180000, 8, 24, "bf16"),
         (360000, 8, 23, "bf16"), (1050000, 8, 4, "bf16"), (700000, 8, 3, "f32")]


@pytest.mark.parametrize("T,k,H,dtype", TAILS)
def test_large_tails(T, k, H, dtype):
    """Every word of every place, bit for bit, and none behind the last run."""
    say(f"dispatch T={T} k={k} H={H} {dtype}")
    m, g, E = moe(), torch.Generator("cuda").manual_seed(T + H), 80
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    ids[::3, k // 2:] = E                                    # another shard's
    sid, _, npad = m.align_block(ids, E, 16)
    n, S = int(npad), T * k
    x = torch.randint(-2 ** 31, 2 ** 31 - 1, (T, H), generator=g, device="cuda").int()
    x = (x >> 16).short().view(torch.bfloat16) if dtype == "bf16" else x.view(torch.float32)
    out, ok = sentinel((sid.numel(), H), dtype)
    rows, at = m.dispatch(x, ids, E, sid, npad, out=out)
    torch.cuda.synchronize()
    ok()
    slot = sid[:n].long()
    live = slot < S
    ref = torch.full((S,), -1, dtype=torch.int32, device="cuda")
    ref[slot[live]] = torch.arange(n, device="cuda", dtype=torch.int32)[live]
    assert torch.equal(at.view(-1), ref)
    want = bits(x)[slot.clamp(max=S - 1) // k]
    want[~live] = 0
    lost = int((bits(rows[:n]) != want).any(1).sum())
    assert lost == 0, f"{lost} of {n} rows are not their token's"
    assert bool((rows[n:] == 12345.0).all()), "rows behind the last run were written"
