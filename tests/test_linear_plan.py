"""The rule that picks the FP8 product's kernel, on the host."""
import random

import pytest

import fp8_quantized_lora_amd as fq
from tests.linear_kinds import STREAM_BYTES, STREAMED, WHOLE
from tests.linear_plan import KINDS, plan

# d_in and d_out up to 2^30 and as many 256 x 256 tiles as the call accepts
DIMS = [16, 48, 4096, 11008, 65536, 1 << 20, (1 << 22) - 16, 1 << 22, 1 << 24, (1 << 26) - 16,
        1 << 26, (1 << 26) + 16, 1 << 28, 1 << 30]
ROWS = [1, 2, 15, 16, 17, 31, 32, 33, 64, 100, 128, 257, 4096, 1 << 16, 1 << 20, 1 << 26, 1 << 30]


def accepted(T, d_in, d_out):
    return 2 * ((T + 255) // 256) * ((max(d_in, d_out) + 255) // 256) <= 2 ** 31 - 1


@pytest.mark.parametrize("d_in", [0, 16, 128, 4096, 13824, (1 << 23) + 16])
def test_every_launch_fits_a_grid(d_in):
    """Fewer than 2^32 threads wherever the operands fit the memory (2^39 bytes)."""
    for T in ROWS:
        for d_out in DIMS:
            if not accepted(T, d_in, d_out) or T * d_out + (T + d_out) * d_in > 2 ** 39:
                continue
            p = plan(T, d_in, d_out)
            assert 0 < p.groups * p.threads < 2 ** 32, (T, d_in, d_out, p)


def test_few_tokens_need_no_workspace():
    """Up to 16 tokens, whatever the other sizes: the binding does not ask."""
    for T in (1, 5, 16):
        for d_in in DIMS:
            for d_out in DIMS:
                assert plan(T, d_in, d_out).split == 1
                if accepted(T, d_in, d_out):
                    assert fq.melded_linear_fwd_act_workspace_bytes(T, d_in, d_out) == 0


def test_tested_shapes_reach_their_kernel():
    """The shapes that the GPU tests list for a kernel get it, none is left out, and
    the streamed ones are streamed."""
    for table in (WHOLE, STREAMED):
        for how, shapes in table.items():
            for T, d_in, d_out in shapes:
                assert plan(T, d_in, d_out).how == how, (T, d_in, d_out)
                assert (4 * T * d_out > STREAM_BYTES) == (table is STREAMED)
    assert set(WHOLE) == {"few1", "few2", "split", *KINDS}


def test_streamed_kinds():
    """No other tile is picked for outputs that are streamed."""
    rng, seen = random.Random(4), set()
    for _ in range(60000):
        T = int(2 ** rng.uniform(0, 26))
        d_out = int(2 ** rng.uniform(0, 22)) * 16
        if 4 * T * d_out > STREAM_BYTES:
            seen.add(plan(T, int(2 ** rng.uniform(0, 12)) * 16, d_out).how)
    assert seen - {"few1"} <= set(STREAMED), seen - set(STREAMED)
