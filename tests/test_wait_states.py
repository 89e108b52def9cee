"""Wait states that inline asm has to bring along, checked over the library's
own GPU code: in asm statements the compiler neither sees the instruction nor
inserts what it needs."""
import re

import pytest

from tests import gfx_asm

pytestmark = pytest.mark.skipif(gfx_asm.objdump() is None, reason="no llvm-objdump")


def direct_loads():
    for name, ins in gfx_asm.functions().items():
        for k, i in enumerate(ins):
            if re.match(r"global_load_lds_|buffer_load_.*_lds", i.op) or "lds" in i.args:
                yield name, ins, k


def test_direct_loads_wait_for_m0():
    """A load into LDS takes its LDS address from m0, which a scalar instruction
    must have written a wait state before (gfx9's rule for memory instructions
    with LDS destinations)."""
    bad, seen = [], 0
    for name, ins, k in direct_loads():
        seen += 1
        if any(i.op.startswith("s_") and i.args and i.args[0] == "m0"
               for i in gfx_asm.before(ins, k, 1)):
            bad.append((name, str(ins[k])))
    assert seen > 100
    assert not bad, f"{len(bad)} of {seen} loads, the first: {bad[0]}"


def test_direct_loads_wait_for_their_base():
    """A scalar base address written by a vector instruction (readfirstlane) must
    lie five wait states back."""
    bad = []
    for name, ins, k in direct_loads():
        base = gfx_asm.registers(" ".join(ins[k].args), "s")
        for i in gfx_asm.before(ins, k, 5):
            if i.op.startswith("v_") and i.args and gfx_asm.registers(i.args[0], "s") & base:
                bad.append((name, str(ins[k]), str(i)))
    assert not bad, bad[0]


# A product of 16 x 16 x 128 takes eight passes; its result may be read or written
# by others four wait states after them at the earliest.  What a vector
# instruction wrote is an operand two wait states later.
RESULT, OPERAND = 12, 2


def product_faults(ins):
    """Where an instruction touches a product's result too early, or a product its
    operands, as text."""
    for k, i in enumerate(ins):
        if not i.op.startswith("v_mfma"):
            continue
        result = gfx_asm.registers(i.args[0])
        walk = gfx_asm.after(ins, k, RESULT)
        for j, waited in walk:
            if not gfx_asm.registers(" ".join(j.args)) & result:
                continue
            onto = (j.op.startswith("v_mfma")                 # accumulates onto the same
                    and gfx_asm.registers(j.args[0]) == gfx_asm.registers(j.args[3]) == result
                    and not gfx_asm.registers(" ".join(j.args[1:3])) & result)
            if not onto:
                yield f"{i}; after {waited}: {j}"
            walk.send(True)
        operands = gfx_asm.registers(" ".join(i.args[1:4]))
        for j in gfx_asm.before(ins, k, OPERAND):
            if (j.op.startswith("v_") and not j.op.startswith("v_mfma") and j.args
                    and gfx_asm.registers(j.args[0]) & operands):
                yield f"{i}; before: {j}"


def test_asm_products_are_left_alone():
    """The tiles of four waves issue their products in asm."""
    seen = 0
    for name, ins in gfx_asm.functions().items():
        if "linear_act_pipe" in name:
            seen += sum(i.op.startswith("v_mfma") for i in ins)
            bad = list(product_faults(ins))
            assert not bad, (name, len(bad), bad[0])
    assert seen > 1000


MFMA = "v_mfma_f32_16x16x128_f8f6f4 a[0:3], v[0:7], v[8:15], a[0:3]"


def listing(*lines):
    """A disassembly of those instructions, four bytes each; "-> n" branches to number n."""
    out = ["0000000000001000 <f>:"]
    for n, text in enumerate(lines):
        text, _, to = text.partition(" -> ")
        where = f" <f+{int(to) * 4:#x}>" if to else ""
        out.append(f"\t{text} // {0x1000 + 4 * n:012X}: 00000000{where}")
    return gfx_asm.parse("\n".join(out))["f"]


@pytest.mark.parametrize("lines, faults", [
    ([MFMA, "s_nop 10", "v_accvgpr_read_b32 v20, a3"], 1),
    ([MFMA, "s_nop 11", "v_accvgpr_read_b32 v20, a3"], 0),
    ([MFMA, "v_accvgpr_write_b32 a1, v20"], 1),
    ([MFMA, MFMA, "s_nop 15", "v_accvgpr_read_b32 v20, a0"], 0),
    ([MFMA, "v_mfma_f32_16x16x128_f8f6f4 a[4:7], v[0:7], a[0:7], a[4:7]"], 1),
    ([MFMA, "v_mfma_f32_16x16x128_f8f6f4 a[2:5], v[0:7], v[8:15], a[2:5]"], 1),
    # along a branch, backward, and past one that is taken
    (["v_accvgpr_read_b32 v20, a2", "s_nop 3", MFMA, "s_cbranch_scc1 65532 -> 0", "s_endpgm"], 1),
    (["v_accvgpr_read_b32 v20, a2", "s_nop 3", MFMA, "s_branch 1 -> 5",
      "v_accvgpr_read_b32 v20, a2", "s_endpgm"], 0),
    (["v_mov_b32_e32 v9, v30", MFMA], 1),
    (["v_mov_b32_e32 v9, v30", "s_nop 0", MFMA], 1),
    (["v_mov_b32_e32 v9, v30", "s_nop 1", MFMA], 0),
    (["v_mov_b32_e32 v16, v9", MFMA], 0),
])
def test_the_check_finds_them(lines, faults):
    assert len(list(product_faults(listing(*lines)))) == faults
