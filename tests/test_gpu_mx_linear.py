"""melded_linear_fwd_mxfp4 against the formula in float64, every element, for each of
its kernels.

Tolerance (u = 2^-24): a product of two FP4 codes is a multiple of 1/4 of at most 36, so
the eight that the matrix core adds at a time are exact, and so is a block's power of
two; their sums are float32's, (d_in / 8 + 2) u sum |x w|.  Bias, activation and residual
as in tests/test_gpu_linear_kinds.py: 4 u |z| for the bias, 16 u |z| (and 6.2e-6 |z|
Phi(-|z|) for gelu rounded to bfloat16) for the activation, whose slope is at most 1.2, u |y|
for the residual; then half a step of the output's type."""
import math

import numpy as np
import pytest
import torch

from tests import mx_ref as ref
from tests.gpu_util import announce, host
from tests.loss_mx_plan import mx
from tests.test_gpu_linear_kinds import act_ref, held

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8
ACTS = ("gelu", "none", "silu", "relu", "gelu_tanh")

# (T, d_in, d_out): one K step of 256 and parts of one, whole and ragged ones, an even
# and an odd number, more than the rings of loads hold; ragged rows and columns
KINDS = {
    "few1": [(1, 32, 16), (3, 160, 1040), (16, 2592, 528), (7, 10272, 112), (1, 256, 4112)],
    "few2": [(17, 32, 272), (29, 288, 1040), (32, 2592, 528), (23, 10272, 112)],
    "32x64": [(33, 32, 144), (33, 224, 144), (61, 256, 144), (33, 544, 144), (95, 768, 144),
              (33, 1280, 144), (33, 2592, 144), (33, 6176, 144)],
    "64": [(33, 32, 16512), (33, 256, 16512), (33, 544, 16528), (33, 768, 16544),
           (33, 1312, 16512), (33, 2080, 8256)],
    "128": [(1810, 32, 4128), (1810, 256, 4128), (200, 544, 24768), (200, 768, 28896),
            (200, 1312, 14448), (65, 2080, 22704), (65, 4128, 22704)],
    "256x128": [(700, 32, 16512), (700, 256, 16512), (513, 544, 20640), (513, 768, 20640),
                (513, 1312, 20640), (513, 2080, 20640), (129, 4128, 22704)],
    "split": [(129, 27648, 528), (66, 24576, 1040), (100, 20512, 784)],
}


def operand(fq, x):
    q = torch.empty((x.shape[0], x.shape[1] // 2), dtype=U8, device="cuda")
    e = torch.empty(fq.mxfp4_scales_shape(*x.shape), dtype=U8, device="cuda")
    fq.mxfp4_quantize(x, q, e)
    v = torch.empty(x.shape, device="cuda")
    fq.mxfp4_dequantize(q, e, v)
    return q, e, v.double()


def check(fq, T, d_in, d_out, dtype, act, use_bias, use_res, keep_z, in_place=False):
    announce(f"melded_linear_fwd_mxfp4 T={T} d_in={d_in} d_out={d_out} {dtype} {act} "
             f"bias={use_bias} residual={use_res} z={keep_z}")
    g = torch.Generator(device="cuda")
    g.manual_seed(T + d_in)
    rn = lambda *s: torch.empty(s, device="cuda").normal_(generator=g)  # noqa: E731
    # blocks of very different sizes, so that every exponent counts
    x = rn(T, d_in) * torch.exp2(torch.randint(-3, 4, (T, d_in // 32, 1), generator=g,
                                               device="cuda").float()).expand(
        T, d_in // 32, 32).reshape(T, d_in)
    w = rn(d_out, d_in) * d_in ** -0.5 * torch.exp2(torch.randint(
        -3, 3, (d_out, d_in // 32, 1), generator=g, device="cuda").float()).expand(
        d_out, d_in // 32, 32).reshape(d_out, d_in)
    (xq, xe, xv), (wq, we, wv) = operand(fq, x), operand(fq, w)
    bias, res = rn(d_out) * 0.3, rn(T, d_out).to(dtype)
    new = lambda: torch.full((T, d_out), float("nan"), dtype=dtype, device="cuda")  # noqa: E731
    y, z = new(), new()
    r0 = res.double()
    if in_place:
        y = res
    fq.melded_linear_fwd_mxfp4(xq, xe, wq, we, y, bias=bias if use_bias else None, act=act,
                               residual=res if use_res else None, z=z if keep_z else None)
    zr = xv @ wv.T
    tol = (xv.abs() @ wv.abs().T).mul_((d_in / 8 + 2) * U)
    tol += zr.abs() * (4 * U)
    if use_bias:
        zr += bias.double()
        tol += zr.abs() * (4 * U)
    if keep_z:
        held(z, zr, tol.clone(), dtype, "z")
    yr = act_ref(zr, act)
    if act != "none":
        tol = tol * 1.2 + 16 * U * zr.abs()
        if act == "gelu" and dtype == BF16:
            tol += 6.2e-6 * zr.abs() * 0.5 * torch.erfc(zr.abs() / math.sqrt(2))
    if use_res:
        yr = yr + r0
        tol = tol + U * yr.abs()
    held(y, yr, tol, dtype, "y")


CASES = [(k, *s, i) for k, v in KINDS.items() for i, s in enumerate(v)]


@pytest.mark.parametrize("kind, T, d_in, d_out, i", CASES)
def test_every_kernel(gpu_lib, kind, T, d_in, d_out, i):
    assert mx(T, d_in, d_out) == kind
    check(gpu_lib, T, d_in, d_out, (F32, BF16)[i % 2], ACTS[i % 5], i % 2 == 0, i % 3 == 0,
          i % 3 != 2)
    check(gpu_lib, T, d_in, d_out, (BF16, F32)[i % 2], ACTS[(i + 2) % 5], i % 2 == 1, i % 3 != 0,
          i % 3 == 2)


@pytest.mark.parametrize("T", [1, 5, 40, 300])
@pytest.mark.parametrize("act", ACTS)
def test_activations_and_a_residual_in_place(gpu_lib, T, act):
    check(gpu_lib, T, 96, 208, BF16, act, True, True, True, in_place=True)


def test_codes_of_another_program(gpu_lib):
    """Operands laid out by the documented rule, not by mxfp4_quantize: random codes and
    exponents, among them the smallest and NaN, which stays in its row."""
    rng = np.random.default_rng(3)
    T, d_in, d_out = 20, 320, 48
    xc, wc = rng.integers(0, 16, (T, d_in)), rng.integers(0, 16, (d_out, d_in))
    xe, we = rng.integers(-9, 9, (T, d_in // 32)), rng.integers(-9, 9, (d_out, d_in // 32))
    xe[3], xe[5, 2] = -127, 128
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a.astype(np.uint8))).cuda()  # noqa: E731
    y = torch.empty((T, d_out), device="cuda")
    for rows in (T, 16):                            # two kernels
        gpu_lib.melded_linear_fwd_mxfp4(dev(ref.pack4(xc[:rows])), dev(ref.pack_exponents(xe[:rows])),
                                        dev(ref.pack4(wc)), dev(ref.pack_exponents(we)), y[:rows])
        xv, wv = ref.decode(xc[:rows], xe[:rows], "fp4"), ref.decode(wc, we, "fp4")
        want, got = xv @ wv.T, host(y[:rows]).astype(np.float64)
        assert np.isnan(got[5]).all() and np.isnan(want[5]).all()
        keep = np.arange(rows) != 5
        S = np.abs(xv[keep]) @ np.abs(wv).T
        assert np.all(np.abs(got[keep] - want[keep]) <= (d_in / 8 + 3) * U * S + 1e-40)


def test_empty_sizes(gpu_lib):
    """No tokens, no outputs; an empty sum is 0."""
    u8 = lambda *s: torch.zeros(s, dtype=U8, device="cuda")  # noqa: E731
    e = lambda r, k: u8(*gpu_lib.mxfp4_scales_shape(r, k))  # noqa: E731
    y = torch.empty((0, 32), device="cuda")
    gpu_lib.melded_linear_fwd_mxfp4(u8(0, 32), e(0, 64), u8(32, 32), e(32, 64), y)
    gpu_lib.melded_linear_fwd_mxfp4(u8(4, 32), e(4, 64), u8(0, 32), e(0, 64),
                                    torch.empty((4, 0), device="cuda"))
    for T in (4, 40, 400):
        y = torch.full((T, 32), float("nan"), device="cuda")
        gpu_lib.melded_linear_fwd_mxfp4(u8(T, 0), e(T, 0), u8(32, 0), e(32, 0), y,
                                        bias=torch.arange(32.0, device="cuda"))
        assert torch.equal(y, torch.arange(32.0, device="cuda").expand(T, 32))
