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
