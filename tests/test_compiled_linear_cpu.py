"""The matrix instructions that the bf16 tiles of moe_linear write in inline assembly are unknown to
the compiler's hazard recogniser, so what it emitted around them is checked here, in the library
as it is built (no GPU needed): a vector instruction that writes an operand is two wait states
ahead of the product, and nothing else touches a product's sums before it has written them."""
import os
import re
import shutil
import struct
import subprocess

import pytest

m = pytest.importorskip("moe_expert_ffn_router_amd")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
OBJDUMP = os.path.join(os.path.dirname(os.path.dirname(HIPCC)), "llvm", "bin", "llvm-objdump")
OPERAND_STATES = 2   # from a vector instruction's result to a product that reads it
RESULT_STATES = 18   # from a product to what else reads or writes its sums (16 passes and two)


def code_objects(path):
    """The gfx950 code objects of a library."""
    data = open(path, "rb").read()
    at = -1
    while (at := data.find(b"__CLANG_OFFLOAD_BUNDLE__", at + 1)) >= 0:
        count, = struct.unpack_from("<Q", data, at + 24)
        entry = at + 32
        for _ in range(count):
            first, size, length = struct.unpack_from("<QQQ", data, entry)
            name = data[entry + 24:entry + 24 + length]
            entry += 24 + length
            if name.endswith(b"gfx950"):
                yield data[at + first:at + first + size]


def registers(operand):
    """The vector registers that an operand names."""
    found = re.fullmatch(r"([va])\[(\d+):(\d+)\]", operand)
    if found:
        return {(found[1], i) for i in range(int(found[2]), int(found[3]) + 1)}
    found = re.fullmatch(r"([va])(\d+)", operand)
    return {(found[1], int(found[2]))} if found else set()


class Instruction:
    def __init__(self, text, address, target):
        words = text.split(None, 1)
        self.text, self.name, self.address, self.target = text, words[0], address, target
        rest = re.split(r",\s*(?![^\[]*\])", words[1]) if len(words) > 1 else []
        self.operands = [registers(o.strip().split(" ")[0]) for o in rest]
        self.states = int(words[1]) + 1 if self.name == "s_nop" else 1
        self.product = self.name.startswith("v_mfma")
        # what a vector instruction writes (comparisons write scalars, swaps both operands)
        self.writes = set()
        if self.name.startswith("v_") and self.operands:
            self.writes = self.operands[0] | (self.operands[1] if "swap" in self.name else set())
        self.touches = set().union(*self.operands)


def parse(lines):
    """Instructions of a function's listing and, of each, those that may come right before it."""
    code = []
    for line in lines:
        text, _, comment = line.partition("// ")
        if not re.match(r"[0-9A-F]{12,}:", comment):       # a label, the padding behind the code
            continue
        address = int(comment.split(":")[0], 16)
        target = re.search(r"<\S+?(?:\+0x([0-9a-f]+))?>", comment)
        code.append(Instruction(text.strip(), address,
                                int(target[1] or "0", 16) if target else None))
    place = {i.address - code[0].address: n for n, i in enumerate(code)}
    before = [[] for _ in code]
    for n, i in enumerate(code):
        if i.name not in ("s_branch", "s_endpgm", "s_setpc_b64") and n + 1 < len(code):
            before[n + 1].append(n)
        if i.target is not None and "branch" in i.name:
            before[place[i.target]].append(n)
    return code, before


def hazards(lines):
    """What stands too close to a product: (instruction, product) texts; and how many products."""
    code, before = parse(lines)

    def back(n, limit):
        """The instructions fewer than `limit` wait states ahead of n, on any path."""
        best, todo = {}, [(p, 0) for p in before[n]]
        while todo:
            p, states = todo.pop()
            if states >= limit or best.get(p, limit) <= states:
                continue
            best[p] = states
            todo += [(q, states + code[p].states) for q in before[p]]
        return best

    found = []
    for n, i in enumerate(code):
        if i.product:
            reads = set().union(*i.operands[1:4])
            found += [(code[p].text, i.text) for p in back(n, OPERAND_STATES)
                      if not code[p].product and code[p].writes & reads]
        elif i.touches:
            found += [(i.text, code[p].text) for p in back(n, RESULT_STATES)
                      if code[p].product and code[p].operands[0] & i.touches]
    return found, sum(i.product for i in code)


def test_built_tiles():
    if shutil.which(OBJDUMP) is None:
        pytest.skip(f"no {OBJDUMP}")
    kernels = 0
    for blob in code_objects(m.LIB_PATH):
        if b"linear11tile_kernel" not in blob:
            continue
        listing = subprocess.run([OBJDUMP, "-d", "/dev/stdin"], input=blob, check=True,
                                 stdout=subprocess.PIPE).stdout.decode()
        for function in re.split(r"\n(?=[0-9a-f]{16} <)", listing):
            head, _, body = function.partition("\n")
            # <MI, NI, gated, operands' type, outputs' type>: t is unsigned short, bf16
            shape = re.search(r"linear11tile_kernelILi(\d+)ELi(\d+)ELb[01]Et[tf]E", head)
            if not shape:
                continue
            kernels += 1
            found, products = hazards(body.splitlines())
            # two steps of the loop at least
            assert products >= 2 * int(shape[1]) * int(shape[2]), head
            assert not found, (head, found[:4])
    assert kernels == 24


def listing(*texts):
    return [f"\t{t} // {0x1000 + 8 * n:016X}: 00000000" + (" <f+0x8>" if "branch" in t else "")
            for n, t in enumerate(texts)]


PRODUCT = "v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[8:11], a[0:3]"


@pytest.mark.parametrize("texts,clean", [
    (["v_mov_b32_e32 v4, v0", PRODUCT], False),
    (["v_mov_b32_e32 v4, v0", "s_nop 0", PRODUCT], False),
    (["v_mov_b32_e32 v4, v0", "s_nop 1", PRODUCT], True),
    (["v_mov_b32_e32 v12, v4", PRODUCT], True),
    (["v_accvgpr_write_b32 a2, 0", PRODUCT], False),
    (["v_permlane32_swap_b32_e32 v0, v9", PRODUCT], False),
    (["ds_read_b128 v[4:7], v0", "s_waitcnt lgkmcnt(0)", PRODUCT], True),
    # around a loop: its last instruction comes before its first
    (["s_nop 0", PRODUCT, "v_add_u32_e32 v11, 1, v11", "s_cbranch_scc1 65533", "s_endpgm"], False),
    (["s_nop 0", PRODUCT, "v_add_u32_e32 v12, 1, v12", "s_cbranch_scc1 65533", "s_endpgm"], True),
    ([PRODUCT, "v_accvgpr_read_b32 v0, a3"], False),
    ([PRODUCT, "s_nop 15", "v_accvgpr_read_b32 v0, a3"], False),
    ([PRODUCT, "s_nop 15", "s_nop 15", "v_accvgpr_read_b32 v0, a3"], True),
    ([PRODUCT, "ds_write_b128 v0, a[0:3]"], False),
    ([PRODUCT, PRODUCT], True)])
def test_the_check_sees_mistakes(texts, clean):
    found, _ = hazards(listing(*texts))
    assert (not found) == clean, found
