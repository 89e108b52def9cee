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
