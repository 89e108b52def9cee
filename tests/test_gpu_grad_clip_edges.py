"""grad_clip where max_norm / (norm + eps) is no number: an infinite max_norm
with an infinite norm, and 0 / 0."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan
BF16 = torch.bfloat16


def tensors(bad=None):
    g = torch.Generator().manual_seed(2)
    t = [torch.randn(5000, generator=g).cuda(), torch.randn(77, generator=g).to(BF16).cuda()]
    if bad is not None:
        t[0][4321] = bad
    return t


def clip(fq, grads, max_norm, apart, **kw):
    norm = torch.full((1,), 5.0, device="cuda")
    out = [torch.full_like(t, 9.0) for t in grads] if apart else grads
    fq.grad_clip(grads, max_norm, norm, out=out if apart else None, **kw)
    return float(norm), out


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("bad", [INF, -INF])
def test_no_limit_and_an_infinity(gpu_lib, bad, apart):
    """The norm is recorded, nothing is scaled."""
    want = tensors(bad)
    norm, out = clip(gpu_lib, tensors(bad), INF, apart)
    assert norm == INF and all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("max_norm", [INF, 1.0, 0.0])
def test_nan(gpu_lib, max_norm, apart):
    norm, out = clip(gpu_lib, tensors(NAN), max_norm, apart)
    assert math.isnan(norm) and all(torch.isnan(t).all() for t in out)


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("max_norm", [0.0, 1.0, INF])
def test_zeros_without_eps(gpu_lib, max_norm, apart):
    norm, out = clip(gpu_lib, [torch.zeros_like(t) for t in tensors()], max_norm, apart, eps=0.0)
    assert norm == 0.0 and not any(t.any() for t in out)


@pytest.mark.parametrize("apart", [False, True])
def test_a_limit_and_an_infinity(gpu_lib, apart):
    """coef is 0: every finite element, and the infinite one 0 * inf."""
    norm, out = clip(gpu_lib, tensors(INF), 3.0, apart)
    assert norm == INF and torch.isnan(out[0][4321])
    out[0][4321] = 0.0
    assert not any(t.any() for t in out)


def test_more_tensors_than_a_launch_names(gpu_lib):
    """The same through the table in the workspace."""
    for bad, max_norm, want in ((INF, INF, "same"), (NAN, INF, "nan"), (0.0, 0.0, "zero")):
        grads = [torch.ones(3 + i, device="cuda") for i in range(300)]
        if bad == 0.0:
            [t.zero_() for t in grads]
        else:
            grads[200][1] = bad
        keep = [t.clone() for t in grads]
        clip(gpu_lib, grads, max_norm, False, eps=0.0)
        for t, k in zip(grads, keep):
            assert (torch.isnan(t).all() if want == "nan" else torch.equal(t, k)), want
