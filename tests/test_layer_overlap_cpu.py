"""The operators around the FFN refuse outputs that share a byte with an operand which other
workgroups of the launch still read. Fake device addresses: each call here is refused on the
host before any HIP call (no GPU needed)."""
import pytest

m = pytest.importorskip("moe_expert_ffn_router_amd")
lib = m.lib
UNSUP = 5
F32, BF16 = 0, 1
# operands of a call, a GiB apart
A, B, C, D, E, F, G, H, J, K = ((i + 1) << 30 for i in range(10))


def touching(at, operand_bytes, out_bytes):
    """Addresses for an output of out_bytes that shares 16 bytes or more with the operand."""
    return {at, at + operand_bytes - 16, at - out_bytes + 16}


def norm_in(x=A, res=B, w=C, T=4, H=64, ro=D, out=E):
    return lib.moe_norm_in(x, res, w, 1.0, 1e-6, T, H, BF16, ro, out, None)


def test_norm_in_outputs_apart_from_the_weight():
    # rows of 64 bf16: 512 bytes of outputs, 256 of weights
    for at in touching(C, 256, 512):
        assert norm_in(out=at) == UNSUP and norm_in(ro=at) == UNSUP
        assert norm_in(out=at, res=None, ro=None) == UNSUP


def norm_out(y=A, ids=B, wts=C, shared=D, gate=E, res=F, w=G, nw=H, out=J, nxt=K):
    # 64 tokens of two slots, rows of 64 bf16
    return lib.moe_norm_out(y, BF16, ids, wts, shared, gate, res, w, nw, 1.0, 1e-6, 64, 8, 64, 2,
                            BF16, out, nxt, None)


@pytest.mark.parametrize("name,at,size", [("ids", B, 512), ("wts", C, 512), ("gate", E, 256),
                                          ("w", G, 256), ("nw", H, 256)])
def test_norm_out_outputs_apart_from_every_vector(name, at, size):
    for out in touching(at, size, 64 * 64 * 2):
        assert norm_out(out=out) == UNSUP and norm_out(nxt=out) == UNSUP
        if name != "nw":
            assert norm_out(out=out, nw=None, nxt=None) == UNSUP


def test_router_logits_apart_from_the_bias():
    # 64 tokens x 16 experts: 4096 bytes of logits, 64 of bias
    for out in touching(C, 64, 4096):
        assert lib.moe_router_logits(A, BF16, B, BF16, C, 64, 16, 64, out, None) == UNSUP


LORA = dict(S=4, n=3, K=64, N=64, r=16, M=16, ldx=64, ldy=64, ldo=64)


def lora(x=A, a=B, b=C, scale=D, sid=E, ba=F, npad=G, ws=H, wsb=1 << 20, y=J, out=K, **sizes):
    s = {**LORA, **sizes}
    return lib.moe_lora_add(x, F32, s["ldx"], a, b, scale, sid, ba, npad, s["S"], s["n"], s["K"],
                            s["N"], s["r"], s["M"], ws, wsb, y, F32, s["ldy"], out, s["ldo"],
                            None)


# factors 3 x 16 x 64 bf16; lists of round_up(4 + 3 x 15, 16) = 64 rows
LORA_OPERANDS = [("a", B, 6144), ("b", C, 6144), ("scale", D, 12), ("sid", E, 256), ("ba", F, 16),
                 ("npad", G, 4)]


@pytest.mark.parametrize("name,at,size", LORA_OPERANDS)
def test_lora_out_apart_from_factors_and_lists(name, at, size):
    for out in touching(at, max(size, 16), 1024):
        assert lora(out=out) == UNSUP
        assert lora(out=out, y=out) == UNSUP                 # in place
    # the last of 4 rows of a column slice, 4096 bytes apart
    assert lora(out=at - 3 * 4096, ldo=1024) == UNSUP
    assert lora(out=at - 3 * 4096 - 240, ldo=1024) == UNSUP


def test_lora_workspace_apart_from_every_operand():
    used = lib.moe_lora_workspace_bytes(4, 3, 64, 16, 16)
    assert used % 256 == 0 and used > 0
    for name, at, size in LORA_OPERANDS + [("x", A, 1024), ("y", J, 1024), ("out", K, 1024)]:
        for ws in {at, at - used + 256, at + (size - 1) // 256 * 256}:
            assert lora(ws=ws) == UNSUP, (name, hex(ws - at))
    # in place, and in a row of a strided operand other than the first
    assert lora(ws=J, y=J, out=J) == UNSUP
    for name, ld in (("x", "ldx"), ("y", "ldy"), ("out", "ldo")):
        at = {"x": A, "y": J, "out": K}[name]
        assert lora(ws=at + 3 * 4096, **{ld: 1024}) == UNSUP, name
