"""linear_cross_entropy_bwd into float32: its logits are the forward's, of products of codes as
float16 summed in float32, and its probabilities two float16 numbers.  Against the
definition in float64, every element, and the float32 gradient of the layer.

Tolerances (u = 2^-24).  A logit is off by (d / 4 + 8) u sum |x w| / s, the scale's three
roundings and the fused step with lse by 4 u |z| + 4 u |lse|, the base-2 argument's own by u
of it, which is 15 + 1.45 |z - lse| at most, p by expm1 of all that and 4 u of itself for the
exponential.  The target's logit is summed apart: a lane adds 16 products of each 1024
codes, one rounding each, and the wave's sum is six more; its expm1 is off by 4 u.  G is the
sum of two float16 numbers: 2^-11 of what 2^-11 leaves, and 2^-40 absolutely (half the
smallest step, 2^-25, under the factor of 2^15).  The products with the weight are summed in
float32, (V / 4 + 8) u of the absolute sum for each of the two numbers, whose sums are added
like the splits' and pieces', 40 u; the row's factor 4 u."""
import math

import pytest
import torch

from tests.gpu_util import announce
from tests.test_gpu_cross_entropy import CASES, Case, within
from tests.test_gpu_cross_entropy_terms import Case as Terms
from tests.test_gpu_cross_entropy_terms import SHAPES as TERMS

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, U8 = torch.float32, torch.uint8


def reference(c, lse):
    """dx and its tolerance, for the lse that the call was given"""
    z = c.xv @ c.wv.T
    S = c.xv.abs() @ c.wv.abs().T
    at = c.target.clamp(min=0)[:, None]
    given = lse.double()[:, None]
    keep = c.target >= 0
    p = torch.exp(z - given)
    onehot = torch.zeros_like(p).scatter_(1, at, 1.0)
    G = p - onehot
    step = 4 * U * z.abs() + 4 * U * given.abs()
    e = S * ((c.d / 4 + 8) * U) + step + (15 + 1.45 * (z - given).abs()) * U
    et = S * ((16 * -(-c.d // 1024) + 6) * U) + step
    EG = torch.where(onehot > 0, p * torch.expm1(et), p * torch.expm1(e)) + 4 * U * G.abs()
    EG += (G.abs() + EG) * 2.0 ** -22 + 2.0 ** -40
    aw = c.wv.abs()
    f = torch.where(keep, c.dloss.double(), torch.zeros_like(c.dloss.double()))[:, None]
    dx = f * (G @ c.wv)
    tol = f.abs() * (EG @ aw + (G.abs() @ aw) * ((2 * (c.V / 4 + 8) + 40) * U)) + 4 * U * dx.abs()
    return dx, tol


def check(fq, c):
    loss, lse = c.forward(fq)
    dx = c.backward(fq, lse, F32)
    ref, tol = reference(c, lse)
    within(dx, ref, tol, "dx")
    return dx, ref


@pytest.mark.parametrize("kinds, shape", CASES)
def test_every_kernel(gpu_lib, kinds, shape):
    announce(f"float32 gradient, T, d, V = {shape}")
    check(gpu_lib, Case(*shape))


@pytest.mark.parametrize("shape", [(17, 48, 77), (129, 16, 65), (300, 64, 999), (700, 4096, 700),
                                   (2100, 512, 9001)])
def test_error_as_a_whole(gpu_lib, shape):
    """rel-L2 2^-19: where the errors are a rounding here and there, not each at its bound,
    p's is some 4 u of |z - lse| and of lse, 2^-20 for those of up to 16; float16
    probabilities or FP8's logits alone would be 2^-13."""
    announce(f"float32 gradient as a whole, T, d, V = {shape}")
    dx, ref = check(gpu_lib, Case(*shape, ignored=0.0))
    assert float((dx.double() - ref).norm()) <= 2.0 ** -19 * float(ref.norm())


@pytest.mark.parametrize("big, shape", [(b, s) for v in TERMS.values() for s in v[-1:]
                                        for b in (64.0, 448.0)])
def test_terms_that_cancel(gpu_lib, big, shape):
    """Logits of four that are left of terms of thousands: the products are exact, so what
    the float32 sums lose is all."""
    announce(f"float32 gradient of cancelling terms, T, d, V = {shape}, {big}")
    check(gpu_lib, Terms(*shape, big=big))


@pytest.mark.parametrize("size", [1.0, 100.0, 1e4])
@pytest.mark.parametrize("sure", [False, True])
@pytest.mark.parametrize("T, d, V", [(64, 16, 3), (300, 272, 999), (700, 1040, 5001)])
def test_large_logits(gpu_lib, T, d, V, sure, size):
    """Logits of up to tens of thousands in exact sums of whole numbers: p is off by what lse
    is, half a step, and by the scale's roundings of z, 8 u of each in all."""
    announce(f"float32 gradient at logits of {size}, T, d, V = {(T, d, V)}")
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = torch.randint(-8, 9, (T, d), generator=g, device="cuda").float()
    w = torch.randint(-8, 9, (V, d), generator=g, device="cuda").float()
    s_x, s_w = torch.full((2, 1), (25 * d ** 0.5 / size) ** 0.5, device="cuda")
    f8 = lambda t: t.to(torch.float8_e4m3fn).view(U8)  # noqa: E731
    z = x.double() @ w.double().T / (s_x.double() * s_w.double())
    target = z.argmax(1) if sure else torch.randint(0, V, (T,), generator=g, device="cuda")
    args = (f8(x), s_x, f8(w), s_w, target)
    loss, lse = torch.empty((2, T), device="cuda")
    dx, dloss = torch.empty((T, d), device="cuda"), torch.ones(T, device="cuda")
    gpu_lib.linear_cross_entropy_fwd(*args, loss, lse)
    gpu_lib.linear_cross_entropy_bwd(*args, lse, dloss, dx)
    p = torch.exp(z - torch.logsumexp(z, 1)[:, None])
    G = p.scatter_add(1, target[:, None], -torch.ones_like(z[:, :1]))
    EG = p * torch.expm1(8 * U * (z.abs() + lse.double().abs()[:, None]) + 32 * U)
    EG += G.abs() * 2.0 ** -21 + 2.0 ** -40
    wv = w.double() / s_w.double()
    tol = EG @ wv.abs() + (G.abs() @ wv.abs()) * ((2 * (V / 4 + 8) + 40) * U)
    within(dx, G @ wv, tol, "dx")


def test_pieces_of_the_vocabulary(gpu_lib):
    """Four pieces of G and of what its rounding leaves, in one workspace of 512 MB."""
    c = Case(16384, 16, 30000)
    assert gpu_lib.linear_cross_entropy_bwd_workspace_bytes(16384, 16, 30000) < 530 << 20
    loss, lse = c.forward(gpu_lib)
    dx = c.backward(gpu_lib, lse, F32)
    rows = slice(16000, 16384)
    part = Case(16384, 16, 30000)
    for name in ("xv", "xm", "target", "dloss"):
        setattr(part, name, getattr(c, name)[rows])
    ref, tol = reference(part, lse[rows])
    within(dx[rows], ref, tol, "dx")


def test_a_layer_of_float32(gpu_lib):
    """LinearCrossEntropy's own gradient, of which float32 is the type unless it is told
    otherwise."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    T, d, V = 200, 96, 700
    x, W = (torch.empty(s, device="cuda").normal_(generator=g) for s in ((T, d), (V, d)))
    head = gpu_lib.LinearCrossEntropy(V, d, T)
    head.init_state(W * d ** -0.5)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    head.forward(x, target)
    dx = head.backward(torch.full((T,), 1 / T, device="cuda"))
    assert dx.dtype == F32
    dec = lambda q, s: q.view(torch.float8_e4m3fn).double() / s.double()  # noqa: E731
    wv = dec(head.wq, head.s_w)
    p = torch.softmax(dec(head.xq, head.s_x) @ wv.T, 1)
    p.scatter_add_(1, target[:, None], -torch.ones_like(p[:, :1]))
    want = p @ wv / T
    assert math.isfinite(float(dx.sum()))
    assert float((dx.double() - want).norm()) <= 2.0 ** -19 * float(want.norm())
