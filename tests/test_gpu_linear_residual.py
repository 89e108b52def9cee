"""melded_linear_fwd_act and melded_linear_fwd_mxfp4 with float32 outputs and a residual,
of its own or y itself, in every kernel that stores them, exactly: the operands are small
whole numbers, whose products, sums, bias and residual float32 holds without rounding."""
import pytest
import torch

from tests.gpu_util import announce
from tests.linear_kinds import WHOLE

pytestmark = pytest.mark.gpu

F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8
SHAPES = [(k, s) for k, v in WHOLE.items() for s in {v[0], v[-1]}]


def whole(g, *shape, most=3):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").float()


def check(fq, T, d_in, d_out, fp4, use_bias, act="relu"):
    g = torch.Generator(device="cuda")
    g.manual_seed(T + d_in + d_out)
    x, w = whole(g, T, d_in, most=2), whole(g, d_out, d_in, most=2)
    bias = whole(g, d_out, most=50) if use_bias else None
    residual = whole(g, T, d_out, most=1000)
    want = x @ w.T                                # at most 4 d_in: whole, below 2^24
    if use_bias:
        want += bias
    if act == "relu":
        want.clamp_(min=0)
    want += residual
    if fp4:
        ops = []
        for t in (x, w):
            q = torch.empty((len(t), d_in // 2), dtype=U8, device="cuda")
            e = torch.empty(fq.mxfp4_scales_shape(len(t), d_in), dtype=U8, device="cuda")
            fq.mxfp4_quantize(t, q, e)
            v = torch.empty_like(t)
            fq.mxfp4_dequantize(q, e, v)
            assert torch.equal(v, t)              # 0, 1 and 2 are codes under any scale here
            ops += [q, e]
        run = fq.melded_linear_fwd_mxfp4
    else:
        one = torch.ones(1, device="cuda")
        ops = []
        for t in (x, w):
            ops += [t.to(torch.float8_e4m3fn).view(U8), one]
        run = fq.melded_linear_fwd_act
    y = torch.full((T, d_out), float("nan"), device="cuda")
    run(*ops, y, bias=bias, act=act, residual=residual)
    assert torch.equal(y, want)
    run(*ops, residual, bias=bias, act=act, residual=residual)
    assert torch.equal(residual, want)


@pytest.mark.parametrize("kind, shape", SHAPES)
def test_fp8(gpu_lib, kind, shape):
    announce(f"residual, {kind} {shape}")
    check(gpu_lib, *shape, fp4=False, use_bias=shape[0] % 2 == 0)


@pytest.mark.parametrize("T, d_in, d_out", [(5, 64, 272), (30, 1056, 528), (33, 128, 144),
                                            (100, 288, 4400), (300, 1056, 8208), (700, 96, 16400),
                                            (2000, 544, 9008), (64, 27648, 528)])
def test_fp4(gpu_lib, T, d_in, d_out):
    announce(f"residual, FP4 {T} x {d_in} x {d_out}")
    check(gpu_lib, T, d_in, d_out, fp4=True, use_bias=T % 2 == 0)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("T, d_out", [(8192, 8208), (4100, 20000)])
def test_more_outputs_than_the_caches_hold(gpu_lib, fp4, T, d_out):
    announce(f"residual, {T} x 64 x {d_out}, FP4 {fp4}")
    check(gpu_lib, T, 64, d_out, fp4, use_bias=True, act="none")
