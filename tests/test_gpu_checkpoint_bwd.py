"""linear_act_bwd_ckpt and layer_norm_bwd_ckpt: the formulas in float64 on the values that
the checkpoint stands for, and the same bits as the calls on those values where each
element is by itself.

Tolerances (u = 2^-24) as in the tests of linear_act_bwd and layer_norm_bwd: dz's slope
off by 16 u (1 + |z|), sums over n terms by (n + 4) u of their absolute sum, then half a
step of the output's type."""
import math

import pytest
import torch

from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
SIZES = [(1, 1), (5, 3), (4, 31), (3, 33), (9, 40), (130, 400), (131, 1027), (300, 77), (700, 64),
         (1100, 1000), (2049, 2056), (2100, 515)]


def saved(fq, x):
    T, d = x.shape
    q = torch.empty((T, d), dtype=U8, device="cuda")
    e = torch.empty(fq.checkpoint_scales_shape(T, d), dtype=U8, device="cuda")
    fq.checkpoint_save(x, q, e)
    v = torch.empty((T, d), device="cuda")
    fq.checkpoint_restore(q, e, v)
    return q, e, v


def within(got, ref, tol, name):
    tol = tol + (ref.abs() + tol) * (torch.finfo(got.dtype).eps / 2) + 1e-37
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (f"{name}: {int(bad.sum())} of {bad.numel()}, worst "
                                 f"{float((err / tol).nan_to_num(nan=math.inf).max()):.3g}")


def slope(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return (0.5 * torch.erfc(-z / math.sqrt(2))
                + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    if act == "silu":
        p = torch.sigmoid(z)
        return p + z * p * torch.sigmoid(-z)
    u2 = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    p = torch.sigmoid(u2)
    return p + z * p * torch.sigmoid(-u2) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)


def draw(T, d, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.empty((T, d), device="cuda").normal_(generator=g)
    x[:, ::17] *= 20                                # blocks with an outlier
    return x, torch.empty((T, d), device="cuda").normal_(generator=g)


@pytest.mark.parametrize("gt", [F32, BF16])
@pytest.mark.parametrize("T, d", SIZES)
def test_act(gpu_lib, T, d, gt):
    x, dy = draw(T, d, T + d)
    dy = dy.to(gt)
    for i, act in enumerate(ACTS):
        announce(f"linear_act_bwd_ckpt T={T} d={d} {act} {gt}")
        q, e, v = saved(gpu_lib, x if i % 2 else x.bfloat16())
        dz = torch.full((T, d), float("nan"), dtype=gt, device="cuda")
        db = torch.full((d,), float("nan"), device="cuda")
        gpu_lib.linear_act_bwd_ckpt(dy, q, e, dz, dbias=db, act=act)
        z, s = v.double(), slope(v.double(), act)
        r = dy.double() * s
        # (in bfloat16 the slope of gelu has 1.6e-6 of its terms)
        rel = 16 * U if gt == F32 else 2e-6
        within(dz, r, dy.double().abs() * rel * (1 + z.abs()), "dz")
        within(db, r.sum(0), (dy.double().abs() * rel * (1 + z.abs())
                              + (T + 4) * U * r.abs()).sum(0), "dbias")
        # the same bits as on the restored values
        dz2 = torch.empty_like(dz)
        gpu_lib.linear_act_bwd(dy, v, dz2, act=act)
        assert torch.equal(dz, dz2)
        # either output alone, and in place
        only = torch.empty_like(db)
        gpu_lib.linear_act_bwd_ckpt(dy, q, e, None, dbias=only, act=act)
        assert torch.equal(only, db)
        inp = dy.clone()
        gpu_lib.linear_act_bwd_ckpt(inp, q, e, inp, act=act)
        assert torch.equal(inp, dz)


@pytest.mark.parametrize("gt", [F32, BF16])
@pytest.mark.parametrize("T, d", SIZES + [(40, 20000), (1030, 18000), (1030, 8200),
                                         (1031, 4096), (1500, 1540), (2500, 513), (4099, 100)])
def test_norm(gpu_lib, T, d, gt):
    announce(f"layer_norm_bwd_ckpt T={T} d={d} {gt}")
    x, dy = draw(T, d, T * 3 + d)
    dy = dy.to(gt)
    x = x if d % 2 else x.bfloat16()
    w = 1 + 0.1 * torch.randn(d, device="cuda")
    mean = x.float().mean(1)
    rstd = ((x.float() - mean[:, None]).square().mean(1) + 1e-5).rsqrt()
    q, e, v = saved(gpu_lib, x)
    nan = lambda *s, t=F32: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
    for weight in (w, None):
        dx, dw, db = nan(T, d, t=gt), nan(d), nan(d)
        gpu_lib.layer_norm_bwd_ckpt(dy, q, e, weight, mean, rstd, dx, dw, db)
        g0, r = dy.double(), rstd.double()[:, None]
        # x - mean is rounded once, its product with rstd again
        xh = (v.double() - mean.double()[:, None]) * r
        exh = 3 * U * xh.abs()
        g = g0 * (1 if weight is None else w.double())
        c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
        e1 = (d + 6) * U * g.abs().mean(1, keepdim=True)
        e2 = ((d + 8) * U * (g * xh).abs()).mean(1, keepdim=True)
        ref = r * (g - c1 - xh * c2)
        tol = r * (4 * U * g.abs() + e1 + xh.abs() * e2 + exh * c2.abs()
                   + 4 * U * (c1.abs() + (xh * c2).abs()))
        within(dx, ref, tol, "dx")
        within(dw, (g0 * xh).sum(0), ((T + 8) * U * (g0 * xh).abs()).sum(0), "dweight")
        within(db, g0.sum(0), ((T + 4) * U * g0.abs()).sum(0), "dbias")
    inp, dw2 = dy.clone(), torch.empty_like(dw)
    gpu_lib.layer_norm_bwd_ckpt(inp, q, e, None, mean, rstd, inp, dw2)
    assert torch.equal(inp, dx) and torch.equal(dw2, dw)


def test_nan_and_infinities_that_were_saved(gpu_lib):
    """A NaN stays in its element, and in its row of layer norm; an infinity is the
    block's largest value, where an activation has its limit."""
    x, dy = draw(6, 96, 5)
    x[1, 40], x[2, 5], x[3, 70] = float("nan"), float("inf"), -float("inf")
    q, e, v = saved(gpu_lib, x)
    dz, db = torch.empty_like(dy), torch.empty(96, device="cuda")
    gpu_lib.linear_act_bwd_ckpt(dy, q, e, dz, dbias=db, act="gelu")
    assert bool(dz[1, 40].isnan()) and int(dz.isnan().sum()) == 1
    assert bool(db[40].isnan()) and int(db.isnan().sum()) == 1
    assert bool(torch.isfinite(v[2:4]).all()) and float(v[2, 5]) >= float(v[2, :32].abs().max())
    mean, rstd, dx = torch.zeros(6, device="cuda"), torch.ones(6, device="cuda"), torch.empty_like(dy)
    gpu_lib.layer_norm_bwd_ckpt(dy, q, e, None, mean, rstd, dx)
    assert bool(dx[1].isnan().all()) and int(dx.isnan().sum()) == 96


def test_no_rows(gpu_lib):
    u8 = lambda *s: torch.empty(s, dtype=U8, device="cuda")  # noqa: E731
    dy, dw, db = torch.empty((0, 48), device="cuda"), *torch.ones((2, 48), device="cuda")
    gpu_lib.linear_act_bwd_ckpt(dy, u8(0, 48), u8(0, 2), dy.clone(), dbias=db, act="gelu")
    assert not bool(db.any())
    db.fill_(1)
    none = torch.empty(0, device="cuda")
    gpu_lib.layer_norm_bwd_ckpt(dy, u8(0, 48), u8(0, 2), None, none, none, dy.clone(), dw, db)
    assert not bool(dw.any()) and not bool(db.any())
