"""Sizes and types that the cross entropy's layer and workspace sizes refuse by themselves, not
by a later call's failure."""
import pytest
import torch

import fp8_quantized_lora_amd as fq


@pytest.mark.parametrize("vocab, d, tokens", [(100, 40, 8), (100, 8, 8), (100, 0, 8), (0, 32, 8),
                                              (100, (1 << 22) + 16, 0), ((1 << 22) + 1, 16, 8),
                                              (100, 32, -1), (100, 16, (1 << 30) + 1)])
def test_layer(vocab, d, tokens):
    with pytest.raises(ValueError, match="must be"):
        fq.LinearCrossEntropy(vocab, d, tokens, device="cpu")


def test_layer_of_the_smallest_sizes():
    head = fq.LinearCrossEntropy(1, 16, 0, device="cpu")
    assert head.dx.shape == (0, 16)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.int64, None])
def test_type_of_the_gradient(dtype):
    with pytest.raises(fq.FalqError, match="dx_dtype: expected float32 or bfloat16"):
        fq.linear_cross_entropy_bwd_workspace_bytes(8, 32, 100, dtype)
