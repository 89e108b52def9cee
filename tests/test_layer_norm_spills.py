"""Layer norm's backward of rows of 8193 to 16384 elements holds two rows in 128 registers a
thread: how much of that the compiler keeps in memory, counted in the built library.  An
address for each piece of a row instead of one for the row was 36 to 49 accesses in
float32, and 4 to 13 % of the time."""
import re

import pytest

from tests import gfx_asm

pytestmark = pytest.mark.skipif(gfx_asm.objdump() is None, reason="no llvm-objdump")


def test_rows_of_16_elements_a_thread():
    seen = 0
    for name, ins in gfx_asm.functions().items():
        # <x's type, dy's type, elements, pieces, threads, streamed, odd width>
        m = re.search(r"ln_bwd_rowsI(f|DF16b)(f|DF16b|S\w*_)Li(\d)ELi(\d)ELi1024ELb\dELb(\d)E", name)
        if not m or int(m[3]) * int(m[4]) != 16:
            continue
        seen += 1
        both = m[1] == m[2] == "f"
        most = (40 if both else 16) if m[5] == "1" else 28 if both else 0
        n = sum(i.op.startswith("scratch_") for i in ins)
        assert n <= most, (name, n)
    assert seen >= 8
