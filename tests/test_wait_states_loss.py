"""The wait states around asm products (tests/test_wait_states.py) in the kernels of the
cross entropy, whose products of 32 x 32 x 16 in float16 take eight passes as well."""
import pytest

from tests import gfx_asm
from tests.test_wait_states import product_faults

pytestmark = pytest.mark.skipif(gfx_asm.objdump() is None, reason="no llvm-objdump")


@pytest.mark.parametrize("kernel", ["loss_pipe", "grads_pipe", "dx_pipe"])
def test_asm_products_are_left_alone(kernel):
    seen = 0
    for name, ins in gfx_asm.functions().items():
        if kernel in name:
            seen += sum(i.op.startswith("v_mfma") for i in ins)
            bad = list(product_faults(ins))
            assert not bad, (name, len(bad), bad[0])
    assert seen > 100
