"""FP4 operands on the way back, as their description has it: the product with the upstream
gradient takes the codes of the weight's transpose, and dX = G W.  Whole numbers, whose
codes, products and sums are exact."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8


def operand(fq, x):
    q = torch.empty((x.shape[0], x.shape[1] // 2), dtype=U8, device="cuda")
    e = torch.empty(fq.mxfp4_scales_shape(*x.shape), dtype=U8, device="cuda")
    fq.mxfp4_quantize(x.contiguous(), q, e)
    return q, e


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T, d_in, d_out", [(1, 64, 96), (5, 272 * 2, 128), (30, 528, 1056),
                                            (200, 1040, 800), (700, 4096, 288)])
def test_product_with_the_upstream_gradient(gpu_lib, T, d_in, d_out, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(T + d_in)
    W = torch.randint(-2, 3, (d_out, d_in), generator=g, device="cuda").to(dtype)
    G = torch.randint(-2, 3, (T, d_out), generator=g, device="cuda").to(dtype)
    dx = torch.full((T, d_in), float("nan"), device="cuda")
    gpu_lib.melded_linear_fwd_mxfp4(*operand(gpu_lib, G), *operand(gpu_lib, W.T), dx)
    assert torch.equal(dx, G.float() @ W.float())
