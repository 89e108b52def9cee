"""gelu and its slope in float32 against float64, element by element.

Bounds (u = 2^-24, q = Phi(-|z|), ex = exp(-z^2 / 2), v = -0.4 |z| t with t =
1 / (1 + 0.4 |z|); q = ex P(v), P a polynomial with P(0) = 1/2):
  P   the fit is off by at most 3.9e-8; v carries five roundings (two of them
      the reciprocal's), sup 5 u |v P'(v)| = 6.8e-8; Horner's roundings sum to
      at most 6.1e-8: 1.3e-7 with the places where they are largest apart,
  ex  one step of exp2 (2 u), three roundings of its argument (1.5 z^2 u), the
      product with P (u),
  1 - q for z > 0: u,
so Phi is off by at most E(z) = 1.3e-7 ex + q (3 + 1.5 z^2) u + u [z > 0]; the
value by |z| E and a rounding of its own, the slope Phi + z ex / sqrt(2 pi) by E,
(5 + 1.5 z^2) u of its second term and a rounding of its own.

Where the result is rounded to bfloat16, q = ex t R(t) with t = 1 / (1 + c |z|).  The
value: c = 0.31, R off by at most 4.7e-6 of q, t carries three roundings (two of them
the reciprocal's), which q takes at most 2.6-fold, coefficients and Horner's steps at
most ten times 1.3 u: 6.2e-6 q in place of 1.3e-7 ex.  The slope: c = 0.36, R with its
float32 coefficients off by at most 9.8e-7 of q, t's roundings taken 2.2-fold,
Horner's steps and the product with t 3.7 u: 1.6e-6 q."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
N = 1 << 16


def arguments():
    g = torch.Generator().manual_seed(11)
    z = torch.cat([torch.empty(N // 2).uniform_(-6, 6, generator=g),
                   torch.empty(N // 4).uniform_(-1, 1, generator=g),
                   torch.empty(N // 8).uniform_(-13, 13, generator=g),
                   torch.logspace(-30, 1, N // 8) * (torch.arange(N // 8) % 2 * 2 - 1)])
    z[:4] = torch.tensor([0.0, -0.0, 30.0, -30.0])
    return z


def parts(z):
    a = z.abs()
    return 0.5 * torch.erfc(a / math.sqrt(2)), torch.exp(-z * z / 2)


def phi(z):
    return 0.5 * torch.erfc(-z / math.sqrt(2))


def phi_tol(z):
    q, ex = parts(z)
    return 1.3e-7 * ex + q * (3 + 1.5 * z * z) * U + U * (z > 0)


def phi_tol_short(z, fit):
    q, _ = parts(z)
    return q * (fit + (3 + 1.5 * z * z) * U) + U * (z > 0)


def held(got, ref, tol):
    err = (got.double().cpu() - ref).abs()
    bad = ~(err <= tol + 1e-37)
    assert not bad.any(), f"{int(bad.sum())} outside, worst {float((err / (tol + 1e-37)).max()):.3g}"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1, 20, 40, 700])
def test_value(gpu_lib, T, dtype):
    """z = bias exactly: the codes are zero."""
    z = arguments()
    one = torch.ones(1, device="cuda")
    zero = lambda n: torch.zeros((n, 16), dtype=torch.uint8, device="cuda")  # noqa: E731
    y = torch.empty((T, N), dtype=dtype, device="cuda")
    gpu_lib.melded_linear_fwd_act(zero(T), one, zero(N), one, y, bias=z.cuda(), act="gelu")
    z = z.double()
    ref = z * phi(z)
    phi_off = phi_tol(z) if dtype == torch.float32 else phi_tol_short(z, 6.2e-6)
    tol = z.abs() * phi_off + U * ref.abs()
    if dtype != torch.float32:
        tol = tol + torch.finfo(dtype).eps / 2 * (ref.abs() + tol)
    held(y[0], ref, tol)
    assert torch.equal(y, y[:1].expand(T, N))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_slope(gpu_lib, dtype):
    z = arguments().view(16, -1)
    dz = torch.empty_like(z, device="cuda", dtype=dtype)
    gpu_lib.linear_act_bwd(torch.ones_like(dz), z.cuda(), dz, act="gelu")
    z = z.double()
    second = z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    ref = phi(z) + second
    tol = (phi_tol(z) if dtype == torch.float32 else phi_tol_short(z, 1.6e-6)) + U * ref.abs()
    tol = tol + second.abs() * (5 + 1.5 * z * z) * U
    if dtype != torch.float32:
        tol = tol + torch.finfo(dtype).eps / 2 * (ref.abs() + tol)
    held(dz, ref, tol)
