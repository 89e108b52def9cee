"""Activations and their slopes far out and where z is not finite."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

INF, NAN, BIG = math.inf, math.nan, 3.3e38
ACTS = ["relu", "gelu", "gelu_tanh", "silu"]


def same(got, want):
    """Bit patterns aside, a NaN is a NaN and 0 is -0."""
    return bool(((got == want) | (got.isnan() & want.isnan())).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [1, 40])
def test_values(gpu_lib, T, act, dtype):
    """Infinity stays one, large values are their own activation, the lowest have
    none, a NaN is one.  z = bias: the codes are zero."""
    z = torch.tensor([INF, BIG, 1e20, 100.0, -100.0, -1e20, -BIG, NAN]).repeat(2).cuda()
    want = torch.tensor([INF, BIG, 1e20, 100.0, 0.0, 0.0, 0.0, NAN]).to(dtype).repeat(2)
    one = torch.ones(1, device="cuda")
    zero = lambda n: torch.zeros((n, 16), dtype=torch.uint8, device="cuda")  # noqa: E731
    y = torch.empty((T, 16), dtype=dtype, device="cuda")
    gpu_lib.melded_linear_fwd_act(zero(T), one, zero(16), one, y, bias=z, act=act)
    assert same(y.cpu(), want.expand(T, 16)), y[0]


@pytest.mark.parametrize("dy", [1.0, -3.0])
@pytest.mark.parametrize("zt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ACTS)
def test_slopes(gpu_lib, act, zt, dy):
    """1 and 0 far out, at the infinities too; below 1e-30 is 0 (the slopes' tails at
    -100 are 1e-42 and less).  A NaN's slope is one, but relu's, which is 0."""
    z = torch.tensor([[INF, BIG, 1e30, 1e20, 100.0, -100.0, -1e20, -1e30, -BIG, -INF]]).to(zt)
    want = torch.tensor([[1.0] * 5 + [0.0] * 5])
    dz = torch.empty((1, 10), device="cuda")
    db = torch.empty(10, device="cuda")
    gpu_lib.linear_act_bwd(torch.full_like(dz, dy), z.cuda(), dz, dbias=db, act=act)
    assert bool(((dz.cpu() / dy - want).abs() <= 1e-30).all()), dz
    assert torch.equal(db, dz[0])
    z = torch.full((1, 10), NAN, dtype=zt, device="cuda")
    gpu_lib.linear_act_bwd(torch.full_like(dz, dy), z, dz, act=act)
    assert (not dz.any()) if act == "relu" else dz.isnan().all()
