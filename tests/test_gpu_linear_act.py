"""melded_linear_fwd_act and linear_act_bwd on the GPU against the formulas in
float64, element by element.

Tolerances (u = 2^-24): the product's error is the matrix core's (gemm_bound);
an activation evaluated in float32 is off by at most 16 u |z| plus, for gelu,
the 7.5e-8 of its distribution function times |z|, and carries the product's
error with its slope, at most 1.2; a slope is off by at most 32 u, plus 7.5e-8
for gelu (the argument's rounding, about 4 u of it, times the derivative of
the logistic function, whose product with the argument stays below 0.5)."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_util import announce, gemm_bound

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def half_step(t):
    return torch.finfo(t).eps / 2


def act_ref(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def slope_ref(z, act):
    z = z.clone().requires_grad_(True)
    (g,) = torch.autograd.grad(act_ref(z, act).sum(), z)
    return torch.where(z.detach() > 0, 1.0, 0.0).double() if act == "relu" else g


def value_tol(z, act):
    return z.abs() * ((0.0 if act in ("none", "relu") else 16 * U)
                      + (7.6e-8 if act == "gelu" else 0.0))


def check(got, ref, tol, name):
    got = got.double().cpu()
    assert got.shape == ref.shape
    err = (got - ref).abs()
    bad = ~(err <= tol + 1e-37)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {got.numel()} outside the bound; worst "
                           f"{float((err / (tol + 1e-37)).nan_to_num(nan=np.inf).max()):.3g} of it")


def problem(seed, T, d_in, d_out, dtype):
    g = torch.Generator().manual_seed(seed)

    def quantized(t):
        if t.numel() == 0:
            return t.to(torch.uint8), torch.ones(1)
        s = (448.0 / t.abs().max()).reshape(1)
        return (t * s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s

    xq, s_x = quantized(torch.randn((T, d_in), generator=g))
    wq, s_w = quantized(torch.randn((d_out, d_in), generator=g)
                        * (2.0 / max(d_in, 1)) ** 0.5)
    bias = 0.3 * torch.randn(d_out, generator=g)
    res = torch.randn((T, d_out), generator=g).to(dtype)
    return xq, s_x, wq, s_w, bias, res


def dec(q):
    return q.view(torch.float8_e4m3fn).double()


def reference(p, act, use_bias, use_res):
    xq, s_x, wq, s_w, bias, res = p
    s = float(s_x.double() * s_w.double())
    acc = dec(xq) @ dec(wq).T / s
    tz = torch.from_numpy(gemm_bound(dec(xq).numpy(), dec(wq).numpy(), s, acc.numpy()))
    z = acc + bias.double() if use_bias else acc
    # the scale's three roundings and the bias's fused one
    tz = tz + 4 * U * (acc.abs() + z.abs())
    y = act_ref(z, act)
    ty = 1.2 * tz + value_tol(z, act)
    if use_res:
        y = y + res.double()
        ty = ty + U * y.abs()
    return z, tz, y, ty


def run(fq, p, act, dtype, use_bias=True, use_res=True, keep_z=True, **kw):
    xq, s_x, wq, s_w, bias, res = (t.cuda() for t in p)
    T, n = xq.shape[0], wq.shape[0]
    y, z = (torch.full((T, n), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    fq.melded_linear_fwd_act(xq, s_x, wq, s_w, y, bias=bias if use_bias else None, act=act,
                             residual=res if use_res else None, z=z if keep_z else None, **kw)
    return y, z


SHAPES = [  # (T, d_in, d_out): one token, a few, every tile size, ragged in each dimension
    (1, 16, 16), (1, 512, 256), (1, 400, 1040), (2, 4096, 48), (5, 144, 272), (16, 256, 512),
    (17, 1040, 80), (37, 528, 1008), (64, 384, 128), (65, 2048, 320), (130, 400, 272),
    (200, 112, 1552), (257, 640, 784), (513, 1152, 1280), (1100, 240, 2576), (3000, 128, 2832),
    (3900, 272, 5120), (2304, 160, 8208), (4096, 96, 6416),
    (132, 48, 11008), (387, 48, 10992), (515, 48, 11104), (259, 48, 10928), (386, 48, 12368),
    (35, 112, 8480), (64, 8208, 512), (100, 6160, 784), (40, 13824, 272),     # split over d_in, ragged ends
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,d_in,d_out", SHAPES)
def test_forward(gpu_lib, T, d_in, d_out, dtype):
    act = ACTS[(T + d_in + d_out // 16) % 5]
    announce(f"melded_linear_fwd_act T={T} d_in={d_in} d_out={d_out} {act} {dtype}")
    if d_in > 4096:
        assert gpu_lib.melded_linear_fwd_act_workspace_bytes(T, d_in, d_out) > 0
    p = problem(T + d_in, T, d_in, d_out, dtype)
    z, tz, y, ty = reference(p, act, True, True)
    gy, gz = run(gpu_lib, p, act, dtype)
    check(gz, z, tz + half_step(dtype) * (z.abs() + tz), "z")
    check(gy, y, ty + half_step(dtype) * (y.abs() + ty), "y")


# more outputs, for each of the larger tiles: one K step and part of one, two to
# eleven, an odd and an even number of them, whole and not; ragged rows and columns
LARGE = [
    (579, 16, 11472), (514, 144, 11008), (578, 256, 9808), (517, 384, 10912),      # 128 x 128
    (644, 528, 8224), (643, 784, 8288), (644, 1152, 8304), (650, 1296, 8224),
    (978, 16, 10912), (257, 144, 9856), (258, 384, 9824), (129, 640, 11056),       # eight waves
    (321, 272, 10912), (385, 384, 11824), (322, 528, 11008), (324, 1152, 10928),   # 128 x 192
    (833, 16, 11744), (641, 144, 11936), (642, 256, 12064), (642, 272, 11984),     # 192 x 128
    (643, 384, 11920), (513, 528, 9824), (641, 640, 10928), (520, 784, 9808),
    (515, 1152, 9840), (518, 1296, 9856),
    (1035, 16, 10896), (1028, 144, 10944), (967, 256, 10976), (968, 384, 11088),   # 256 x 128
    (1154, 528, 9808), (977, 640, 11008), (1156, 784, 9760), (1033, 1152, 10896),
    (1293, 16, 10912), (1287, 144, 10960), (1281, 256, 10896), (1298, 384, 11008),  # 128 x 256
    (1300, 528, 11024), (1282, 640, 10896), (1288, 1152, 10896),
    (1039, 1296, 10944), (1031, 2064, 10896), (963, 3088, 10944), (3841, 4096, 4096),  # 256 x 256
    (2690, 784, 6544), (1538, 1296, 10976), (1288, 2064, 11808), (3841, 3584, 5104),   # 256 x 320
]


@pytest.mark.parametrize("T,d_in,d_out", LARGE)
def test_forward_of_many_outputs(gpu_lib, T, d_in, d_out):
    """Every seventh row and the last ones, all columns; the rest is written."""
    p = problem(17, T, d_in, d_out, BF16)
    act = ACTS[(T + d_out // 16) % 5]
    gy, gz = run(gpu_lib, p, act, BF16)
    rows = torch.tensor(sorted({*range(0, T, 7 if T < 1000 else 23), T - 2, T - 1}))
    xq, s_x, wq, s_w, bias, res = p
    z, tz, y, ty = reference((xq[rows], s_x, wq, s_w, bias, res[rows]), act, True, True)
    check(gz.cpu()[rows], z, tz + half_step(BF16) * (z.abs() + tz), "z")
    check(gy.cpu()[rows], y, ty + half_step(BF16) * (y.abs() + ty), "y")
    assert torch.isfinite(gy).all() and torch.isfinite(gz).all()


@pytest.mark.parametrize("T,d_in,d_out", [(3841, 4096, 4096), (3841, 3584, 5104),
                                          (644, 1152, 8304), (1033, 1152, 10896)])
def test_many_outputs_repeat(gpu_lib, T, d_in, d_out):
    """The same bits from every call, float32 too, however the tiles overlap."""
    for dtype in (BF16, F32):
        p = problem(18, T, d_in, d_out, dtype)
        first = run(gpu_lib, p, "silu", dtype)
        for _ in range(4):
            for a, b in zip(first, run(gpu_lib, p, "silu", dtype)):
                assert torch.equal(a, b)


@pytest.mark.parametrize("use_bias,use_res,keep_z", [(False, False, False), (True, False, True),
                                                     (False, True, False)])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,d_in,d_out", [(3, 288, 96), (150, 256, 304)])
def test_forward_parts(gpu_lib, T, d_in, d_out, act, use_bias, use_res, keep_z):
    p = problem(9, T, d_in, d_out, BF16)
    z, tz, y, ty = reference(p, act, use_bias, use_res)
    gy, gz = run(gpu_lib, p, act, BF16, use_bias, use_res, keep_z)
    check(gy, y, ty + half_step(BF16) * (y.abs() + ty), "y")
    if keep_z:
        check(gz, z, tz + half_step(BF16) * (z.abs() + tz), "z")
    else:
        assert torch.isnan(gz).all()                       # left as it was


@pytest.mark.parametrize("T,d_in,d_out", [(1, 4096, 4096), (33, 1024, 2048), (96, 512, 4096),
                                          (1000, 256, 512)])
def test_same_as_the_plain_product(gpu_lib, T, d_in, d_out):
    """No epilogue, float32: the matrix core's sums, so within the same bound
    as melded_linear_fwd; a residual added in place and apart agree bit for
    bit."""
    p = problem(4, T, d_in, d_out, F32)
    gy, _ = run(gpu_lib, p, "none", F32, False, False, False)
    plain = torch.empty_like(gy)
    gpu_lib.melded_linear_fwd(*(t.cuda() for t in p[:4]), plain)
    z, tz, _, _ = reference(p, "none", False, False)
    check(gy, z, tz, "y")
    check(plain, z, tz, "plain")
    apart, _ = run(gpu_lib, p, "silu", F32, True, True, False)
    xq, s_x, wq, s_w, bias, res = (t.cuda() for t in p)
    gpu_lib.melded_linear_fwd_act(xq, s_x, wq, s_w, res, bias=bias, act="silu", residual=res)
    assert torch.equal(res, apart)


@pytest.mark.parametrize("T", [1, 40, 300, 2100])
def test_nan_and_range(gpu_lib, T):
    """A NaN code in row 0 makes that row NaN and no other; codes at +-448
    through a long row stay finite."""
    d_in, d_out = 272, 2064
    xq, s_x, wq, s_w, bias, res = problem(7, T, d_in, d_out, BF16)
    xq[0, 270] = 0x7F
    gy, _ = run(gpu_lib, (xq, s_x, wq, s_w, bias, res), "gelu", BF16, keep_z=False)
    assert torch.isnan(gy[0]).all() and torch.isfinite(gy[1:]).all()
    xq[:], wq[:] = 0x7E, 0xFE                              # 448 and -448
    gy, gz = run(gpu_lib, (xq, s_x, wq, s_w, bias, res), "relu", F32, use_res=False)
    assert torch.isfinite(gz).all() and not gy.any()


def test_empty(gpu_lib):
    """T = 0 and d_out = 0 write nothing; d_in = 0 leaves the bias."""
    for T, d_in, d_out in ((0, 64, 32), (4, 64, 0), (4, 0, 32)):
        p = problem(1, T, d_in, d_out, BF16)
        gy, gz = run(gpu_lib, p, "none", BF16, use_res=False)
        assert gy.shape == (T, d_out)
        if d_in == 0:
            assert torch.equal(gy.cpu(), p[4].to(BF16).expand(T, d_out))


@pytest.mark.parametrize("zt,gt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,d", [(1, 1), (300, 3), (5, 4), (300, 130), (3, 17), (130, 400), (1, 4096), (1003, 1027),
                                 (2050, 264), (40, 11008)])
def test_backward(gpu_lib, T, d, act, zt, gt):
    announce(f"linear_act_bwd T={T} d={d} {act} {zt} {gt}")
    g = torch.Generator().manual_seed(T + d)
    dy = (torch.randn((T, d), generator=g) * 1e-3).to(gt)
    z = (torch.randn((T, d), generator=g) * 3.0).to(zt)
    z.view(-1)[: min(5, z.numel())] = torch.tensor([0.0, 40.0, -40.0, 1e4, -1e4])[: z.numel()].to(zt)
    dz = torch.full((T, d), float("nan"), dtype=gt, device="cuda")
    db = torch.full((d,), float("nan"), device="cuda")
    gpu_lib.linear_act_bwd(dy.cuda(), z.cuda(), dz, dbias=db, act=act)
    ref = dy.double() * slope_ref(z.double(), act)
    tol = dy.double().abs() * ((32 * U if act not in ("none", "relu") else 0.0)
                               + (7.6e-8 if act == "gelu" else 0.0)) + U * ref.abs()
    check(dz, ref, tol + half_step(gt) * (ref.abs() + tol), "dz")
    check(db, ref.sum(0), tol.sum(0) + (T + 8) * U * ref.abs().sum(0), "dbias")
    # dbias alone, in place, and without dbias: the same bits
    alone = torch.full((d,), float("nan"), device="cuda")
    gpu_lib.linear_act_bwd(dy.cuda(), z.cuda(), None, dbias=alone, act=act)
    assert torch.equal(alone, db)
    inp = dy.cuda()
    gpu_lib.linear_act_bwd(inp, z.cuda(), inp, act=act)
    assert torch.equal(inp, dz)
    if act == "none":
        gpu_lib.linear_act_bwd(dy.cuda(), None, inp, act=act)
        assert torch.equal(inp, dz)


@pytest.mark.parametrize("T", [2, 60, 300])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_anywhere_in_a_buffer(gpu_lib, T, dtype):
    """Outputs, residual, bias and z that begin one element into a buffer: the
    bits of aligned ones, and nothing around the outputs changes."""
    d_in, d_out = 272, 144
    p = problem(13, T, d_in, d_out, dtype)
    xq, s_x, wq, s_w, bias, res = (t.cuda() for t in p)

    def at1(v):
        buf = torch.full((v.numel() + 2,), 7.0, dtype=v.dtype, device="cuda")
        buf[1:-1] = v.reshape(-1)
        return buf, buf[1:-1].view(v.shape)

    def run(place):
        y, z, dz = (place(torch.zeros((T, d_out), dtype=dtype, device="cuda")) for _ in range(3))
        db = place(torch.zeros(d_out, device="cuda"))
        gpu_lib.melded_linear_fwd_act(xq, s_x, wq, s_w, y[1], bias=place(bias)[1], act="silu",
                                      residual=place(res)[1], z=z[1])
        gpu_lib.linear_act_bwd(place(res)[1], z[1], dz[1], dbias=db[1], act="silu")
        return y, z, dz, db

    for (buf, v), (_, q) in zip(run(at1), run(lambda v: (None, v.clone()))):
        assert torch.equal(v, q)
        assert float(buf[0]) == 7.0 and float(buf[-1]) == 7.0


@pytest.mark.parametrize("act", ACTS[1:])
def test_slopes_against_differences(gpu_lib, act):
    """dz for dy = 1 against central differences of the activation in float64:
    the quotient is off by h^2 / 6 times the third derivative, at most 2 here."""
    z = torch.linspace(-6, 6, 1608).reshape(3, 536) + 0.00123
    dz = torch.empty((3, 536), device="cuda")
    gpu_lib.linear_act_bwd(torch.ones((3, 536), device="cuda"), z.cuda(), dz, act=act)
    h = 1e-4
    num = (act_ref(z.double() + h, act) - act_ref(z.double() - h, act)) / (2 * h)
    check(dz, num, torch.full_like(num, 34 * U + 7.6e-8 + h * h), "dz")


def test_no_rows(gpu_lib):
    e = torch.empty((0, 48), device="cuda")
    db = torch.full((48,), float("nan"), device="cuda")
    gpu_lib.linear_act_bwd(e, e.clone(), e.clone(), dbias=db, act="silu")
    assert not db.any()


@pytest.mark.parametrize("T", [1, 24, 100, 700])
def test_repeats_other_stream_and_graph(gpu_lib, T):
    """The same bits on another stream, and in three replays of a captured
    graph with eager work between them."""
    d_in, d_out = 656, 1424
    xq, s_x, wq, s_w, bias, res = (t.cuda() for t in problem(30 + T, T, d_in, d_out, BF16))
    dy = torch.randn((T, d_out), device="cuda")
    ws = torch.empty(gpu_lib.linear_act_bwd_workspace_bytes(T, d_out), dtype=torch.uint8,
                     device="cuda")
    new = lambda: [torch.empty((T, d_out), dtype=BF16, device="cuda"),  # noqa: E731
                   torch.empty((T, d_out), dtype=BF16, device="cuda"),
                   torch.empty((T, d_out), device="cuda"), torch.empty(d_out, device="cuda")]

    def both(o, stream=None, w_=None):
        gpu_lib.melded_linear_fwd_act(xq, s_x, wq, s_w, o[0], bias=bias, act="gelu",
                                      residual=res, z=o[1], stream=stream)
        gpu_lib.linear_act_bwd(dy, o[1], o[2], dbias=o[3], act="gelu", ws=w_, stream=stream)

    ref = new()
    both(ref)
    torch.cuda.synchronize()
    side, on_side = torch.cuda.Stream(), new()
    both(on_side, stream=side)
    side.synchronize()
    assert all(torch.equal(a, r) for a, r in zip(on_side, ref))
    out = new()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(out, w_=ws)
    for _ in range(3):
        for t in out:
            t.fill_(float("nan"))
        res.add_(0.25)
        graph.replay()
        torch.cuda.synchronize()
        again = new()
        both(again)
        torch.cuda.synchronize()
        assert all(torch.equal(a, r) for a, r in zip(out, again))
