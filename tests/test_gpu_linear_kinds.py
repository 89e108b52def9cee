"""Every kernel of melded_linear_fwd_act against the formula in float64, every
element of y and z, in float32 and bfloat16, and with outputs that are streamed.

Tolerances (u = 2^-24) as derived in tests/gpu_util.gemm_bound for the product on
the matrix cores; the scale's three roundings and the bias's fused one, 4 u (|acc| +
|z|); an activation in float32 16 u |z| (and 6.2e-6 |z| Phi(-|z|) for gelu rounded to
bfloat16), the product's error with its slope, at most 1.2; the residual's u |y|;
half a step of the output's type."""
import math

import pytest
import torch

from tests.gpu_util import announce
from tests.linear_kinds import STREAMED, WHOLE

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
ACTS = ("gelu", "none", "silu", "relu", "gelu_tanh")


def act_ref(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z) if act == "silu" else z


def codes(g, rows, d):
    """E4M3 codes of normal values, their scale, their values and the largest power
    of two in each eight of a row (gemm_bound)."""
    x = torch.empty((rows, d), device="cuda").normal_(generator=g)
    s = (448.0 / x.abs().max()).reshape(1)
    q = (x * s).clamp(-448, 448).to(torch.float8_e4m3fn)
    v = q.double()
    e = torch.where(v == 0, -6.0, v.abs().clamp(min=2.0 ** -6).log2().floor())
    return q.view(torch.uint8), s, v, torch.exp2(e.view(rows, d // 8, 8).amax(2))


def held(got, ref, tol, dtype, name):
    tol.add_((ref.abs() + tol).mul_(torch.finfo(dtype).eps / 2)).add_(1e-37)
    err = (got.double() - ref).abs_()
    bad = ~(err <= tol)
    n = int(bad.sum())
    assert n == 0, (f"{name}: {n} of {got.numel()}, the first at {bad.nonzero()[0].tolist()}, "
                    f"worst {float((err / tol).nan_to_num(nan=math.inf).max()):.3g} of the bound")


def check(fq, T, d_in, d_out, dtype, act, use_bias, use_res, keep_z):
    announce(f"melded_linear_fwd_act T={T} d_in={d_in} d_out={d_out} {dtype} {act} "
             f"bias={use_bias} residual={use_res} z={keep_z}")
    g = torch.Generator(device="cuda")
    g.manual_seed(T + d_in)
    xq, s_x, xv, xm = codes(g, T, d_in)
    wq, s_w, wv, wm = codes(g, d_out, d_in)
    bias = torch.empty(d_out, device="cuda").normal_(0, 0.3, generator=g)
    res = torch.empty((T, d_out), device="cuda").normal_(generator=g).to(dtype)
    new = lambda: torch.full((T, d_out), float("nan"), dtype=dtype, device="cuda")  # noqa: E731
    y, z = new(), new()
    # activations see values around 1: the product's scale goes into s_w
    s_w = s_w * d_in ** 0.5
    fq.melded_linear_fwd_act(xq, s_x, wq, s_w, y, bias=bias if use_bias else None, act=act,
                             residual=res if use_res else None, z=z if keep_z else None)
    s = float(s_x.double() * s_w.double())
    ref = (xv @ wv.T).div_(s)
    tol = (xm @ wm.T).mul_(7 * 2.0 ** -13 / s)
    tol += (xv.abs() @ wv.abs().T).mul_((d_in / 8 + 2) * U / s)
    tol += ref.abs().mul_(8 * U)
    if use_bias:
        ref += bias.double()
    tol += ref.abs().mul_(4 * U)
    if keep_z:
        held(z, ref, tol.clone(), dtype, "z")
    else:
        assert torch.isnan(z).all()
    tol.mul_(1.2)
    if act not in ("none", "relu"):
        tol += ref.abs().mul_(16 * U)
    if act == "gelu":
        tol += ref.abs() * (torch.erfc(ref.abs() / math.sqrt(2)) * 3.1e-6 if dtype == BF16
                            else 1.3e-7 * torch.exp(-ref * ref / 2))
    ref = act_ref(ref, act)
    if use_res:
        ref += res.double()
        tol += ref.abs().mul_(U)
    held(y, ref, tol, dtype, "y")


def listed(table):
    return [pytest.param(*s, n, id=f"{how}-{s[0]}x{s[1]}x{s[2]}")
            for how, shapes in table.items() for n, s in enumerate(shapes)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T, d_in, d_out, n", listed(WHOLE))
def test_every_kernel(gpu_lib, T, d_in, d_out, n, dtype):
    check(gpu_lib, T, d_in, d_out, dtype, ACTS[(n + (dtype == F32)) % 5], n % 3 != 1, n % 2 == 0,
          n % 4 != 3)


@pytest.mark.parametrize("T, d_in, d_out, n", listed(STREAMED))
def test_streamed_outputs(gpu_lib, T, d_in, d_out, n):
    check(gpu_lib, T, d_in, d_out, BF16, ACTS[n % 5], n % 3 != 1, n % 2 == 0, True)
    torch.cuda.empty_cache()
