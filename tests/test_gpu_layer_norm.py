"""layer_norm_fwd / layer_norm_bwd on the GPU against the formulas in float64,
element by element, and the gradients against central differences.

Tolerances (u = 2^-24, one float32 rounding): a row's sums have at most
D = d / 64 + 16 additions in a chain (64 lanes at least share a row), so a sum
of terms t is off by (D + 2) u sum |t|.  An output in type t adds
finfo(t).eps / 2 of its value."""
import numpy as np
import pytest
import torch

from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def half_step(t):
    return torch.finfo(t).eps / 2


def problem(seed, T, d, xt=F32, gt=F32, offset=0.1, outliers=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, d), generator=g)
    if outliers and d >= 100:
        x[:, torch.randperm(d, generator=g)[: d // 100]] *= 20.0
    x = (x + offset).to(xt)
    dy = (torch.randn((T, d), generator=g) * 1e-3).to(gt)
    w = 1.0 + 0.1 * torch.randn(d, generator=g)
    b = 0.1 * torch.randn(d, generator=g)
    return x, dy, w, b


def ref_fwd(x, w, b, eps):
    x = x.double()
    mu = x.mean(1)
    var = (x - mu[:, None]).square().mean(1)
    rstd = (var + eps) ** -0.5
    xh = (x - mu[:, None]) * rstd[:, None]
    y = xh * (w.double() if w is not None else 1.0) + (b.double() if b is not None else 0.0)
    return y, mu, rstd, xh


def check(got, ref, tol, name):
    got = got.double().cpu()
    assert got.shape == ref.shape
    err = (got - ref).abs()
    bad = ~(err <= tol + 1e-37)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {got.numel()} outside the bound; worst "
                           f"{float((err / (tol + 1e-37)).nan_to_num(nan=np.inf).max()):.3g} of it")


def fwd_tol(x, w, b, y, mu, rstd, xh, yt):
    d = x.shape[1]
    D = d / 64 + 16
    x = x.double()
    dmu = (D + 2) * U * x.abs().mean(1)
    # the mean's error moves the variance by its square only
    rel = (D + 8) * U + (rstd * dmu) ** 2
    aw = w.double().abs() if w is not None else 1.0
    ab = b.double().abs() if b is not None else 0.0
    t = aw * ((rstd * dmu)[:, None] * (1 + 4 * U) + xh.abs() * rel[:, None]) \
        + 3 * U * (aw * xh.abs() + ab)
    return t + half_step(yt) * (y.abs() + t), dmu + U * mu.abs(), rel * rstd


SHAPES = [(1, 1), (4, 2), (3, 3), (6, 4), (7, 5), (9, 6), (3, 7), (5, 8), (1, 4096), (2, 64), (130, 400), (67, 1000), (33, 1027),
          (9, 2048), (40, 4096), (17, 5120), (6, 8192), (5, 8200), (3, 13824), (2, 16384),
          (2, 16392), (2, 20001)]


@pytest.mark.parametrize("xt,yt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward(gpu_lib, T, d, xt, yt):
    announce(f"layer_norm_fwd T={T} d={d} {xt} {yt}")
    x, _, w, b = problem(T * 7 + d, T, d, xt)
    y = torch.full((T, d), float("nan"), dtype=yt, device="cuda")
    mean, rstd = (torch.full((T,), float("nan"), device="cuda") for _ in range(2))
    gpu_lib.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda(), y, mean, rstd)
    ry, rm, rr, xh = ref_fwd(x, w, b, 1e-5)
    ty, tm, tr = fwd_tol(x, w, b, ry, rm, rr, xh, yt)
    check(mean, rm, tm, "mean")
    check(rstd, rr, tr, "rstd")
    check(y, ry, ty, "y")


@pytest.mark.parametrize("weight,bias,stats", [(False, False, True), (True, False, False),
                                               (False, True, False)])
@pytest.mark.parametrize("d", [129, 512])
def test_forward_parts(gpu_lib, weight, bias, stats, d):
    """No weight, no bias, no statistics, each on its own."""
    x, _, w, b = problem(3, 21, d)
    w, b = (w if weight else None), (b if bias else None)
    y = torch.empty((21, d), device="cuda")
    st = [torch.empty(21, device="cuda") for _ in range(2)] if stats else [None, None]
    gpu_lib.layer_norm_fwd(x.cuda(), w.cuda() if weight else None, b.cuda() if bias else None, y,
                           *st, eps=1e-3)
    ry, rm, rr, xh = ref_fwd(x, w, b, 1e-3)
    check(y, ry, fwd_tol(x, w, b, ry, rm, rr, xh, F32)[0], "y")


def test_forward_far_from_zero(gpu_lib):
    """Rows whose mean is 1e4 times their spread, and constant rows: the
    variance is a sum of squared differences, never a difference of squares."""
    x, _, w, b = problem(5, 12, 1536, offset=1e4, outliers=False)
    x[3] = 7.25
    x[4] = 0.0
    y, mean, rstd = torch.empty((12, 1536), device="cuda"), *(torch.empty(12, device="cuda")
                                                              for _ in range(2))
    gpu_lib.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda(), y, mean, rstd)
    ry, rm, rr, xh = ref_fwd(x, w, b, 1e-5)
    ty, tm, tr = fwd_tol(x, w, b, ry, rm, rr, xh, F32)
    check(mean, rm, tm, "mean")
    check(rstd, rr, tr, "rstd")
    check(y, ry, ty, "y")
    assert torch.equal(y[4].cpu(), b)                       # a zero row is the bias


def test_rows_with_nan_and_inf_stay_apart(gpu_lib):
    x, dy, w, b = problem(6, 9, 640)
    x[2, 5], x[7, 600] = float("nan"), float("inf")
    y, mean, rstd = torch.empty((9, 640), device="cuda"), *(torch.empty(9, device="cuda")
                                                            for _ in range(2))
    gpu_lib.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda(), y, mean, rstd)
    dx = torch.empty((9, 640), device="cuda")
    gpu_lib.layer_norm_bwd(dy.cuda(), x.cuda(), w.cuda(), mean, rstd, dx)
    for r in range(9):
        assert bool(torch.isnan(y[r]).all() if r in (2, 7) else torch.isfinite(y[r]).all()), r
        assert bool(torch.isnan(dx[r]).all() if r in (2, 7) else torch.isfinite(dx[r]).all()), r


def ref_bwd(dy, x, w, mean, rstd):
    dy, x = dy.double(), x.double()
    r = rstd.double()[:, None]
    xh = (x - mean.double()[:, None]) * r
    g = dy * w.double() if w is not None else dy
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - c1 - xh * c2)
    d = x.shape[1]
    D = d / 64 + 16
    # x - mean is rounded once, times rstd once: xh is off by 2 u |xh|
    tdx = r * ((D + 4) * U * g.abs().mean(1, keepdim=True)
               + xh.abs() * (D + 8) * U * (g * xh).abs().mean(1, keepdim=True)
               + 8 * U * (g.abs() + c1.abs() + (xh * c2).abs()))
    T = x.shape[0]
    dw, db = (dy * xh).sum(0), dy.sum(0)
    return (dx, dw, db), (tdx, (T + 8) * U * (dy * xh).abs().sum(0),
                          (T + 8) * U * dy.abs().sum(0))


def stats_of(x, eps=1e-5):
    _, mu, rstd, _ = ref_fwd(x, None, None, eps)
    return mu.float(), rstd.float()


@pytest.mark.parametrize("xt,gt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("T,d", SHAPES + [(1500, 96), (700, 1027), (2100, 264), (1025, 1029), (1500, 4096), (1100, 9000), (1030, 3), (1040, 6), (1100, 9001),
                                           (1050, 255)])
def test_backward(gpu_lib, T, d, xt, gt):
    announce(f"layer_norm_bwd T={T} d={d} {xt} {gt}")
    x, dy, w, _ = problem(T * 5 + d, T, d, xt, gt)
    mean, rstd = stats_of(x)
    dx = torch.full((T, d), float("nan"), dtype=gt, device="cuda")
    dw, db = (torch.full((d,), float("nan"), device="cuda") for _ in range(2))
    gpu_lib.layer_norm_bwd(dy.cuda(), x.cuda(), w.cuda(), mean.cuda(), rstd.cuda(), dx, dw, db)
    (rx, rw, rb), (tx, tw, tb) = ref_bwd(dy, x, w, mean, rstd)
    check(dx, rx, tx + half_step(gt) * (rx.abs() + tx), "dx")
    check(dw, rw, tw, "dweight")
    check(db, rb, tb, "dbias")


@pytest.mark.parametrize("T,d", [(50, 515), (50, 768), (1300, 515), (1300, 768), (1050, 8200),
                                 (1030, 8201), (30, 2), (1100, 3)])
def test_backward_parts_and_in_place(gpu_lib, T, d):
    """dx alone, dweight or dbias alone, no weight, dx onto dy: the same bits."""
    x, dy, w, _ = problem(8, T, d)
    mean, rstd = (t.cuda() for t in stats_of(x))
    x, dy, w = x.cuda(), dy.cuda(), w.cuda()
    new = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
    full = [new(T, d), new(d), new(d)]
    gpu_lib.layer_norm_bwd(dy, x, w, mean, rstd, *full)
    for keep in ((0,), (1,), (2,), (1, 2), (0, 2)):
        part = [new(*t.shape) if i in keep else None for i, t in enumerate(full)]
        gpu_lib.layer_norm_bwd(dy, x, w, mean, rstd, *part)
        for i in keep:
            assert torch.equal(part[i], full[i]), (keep, i)
    ones = new(T, d)
    gpu_lib.layer_norm_bwd(dy, x, torch.ones(d, device="cuda"), mean, rstd, ones)
    none = new(T, d)
    gpu_lib.layer_norm_bwd(dy, x, None, mean, rstd, none)
    assert torch.equal(none, ones)
    inp, dw, db = dy.clone(), new(d), new(d)
    gpu_lib.layer_norm_bwd(inp, x, w, mean, rstd, inp, dw, db)
    assert torch.equal(inp, full[0]) and torch.equal(dw, full[1]) and torch.equal(db, full[2])


@pytest.mark.parametrize("T,d", [(40, 129), (40, 640), (1100, 264), (3, 20000)])
@pytest.mark.parametrize("t", [F32, BF16])
def test_rows_anywhere_in_a_buffer(gpu_lib, T, d, t):
    """Rows, parameters and statistics that begin one element into a buffer:
    the bits of aligned ones, and nothing around the outputs changes."""
    x, dy, w, b = problem(31, T, d, t, t)

    def at1(v):
        buf = torch.full((v.numel() + 2,), 7.0, dtype=v.dtype, device="cuda")
        buf[1:-1] = v.reshape(-1).cuda()
        return buf, buf[1:-1].view(v.shape)

    def run(place):
        ins = [place(v) for v in (x, dy, w, b)]
        outs = [place(torch.zeros(s, dtype=dt)) for s, dt in (((T, d), t), ((T,), F32),
                                                              ((T,), F32), ((T, d), t),
                                                              ((d,), F32), ((d,), F32))]
        (_, xv), (_, gv), (_, wv), (_, bv) = ins
        y, m, r, dx, dw, db = (v for _, v in outs)
        gpu_lib.layer_norm_fwd(xv, wv, bv, y, m, r)
        gpu_lib.layer_norm_bwd(gv, xv, wv, m, r, dx, dw, db)
        return outs

    shifted, plain = run(at1), run(lambda v: (None, v.cuda()))
    for (buf, v), (_, p) in zip(shifted, plain):
        assert torch.equal(v, p)
        assert float(buf[0]) == 7.0 and float(buf[-1]) == 7.0


def test_no_rows(gpu_lib):
    """T = 0: nothing but zero gradients of weight and bias."""
    e = torch.empty((0, 24), device="cuda")
    s = torch.empty(0, device="cuda")
    gpu_lib.layer_norm_fwd(e, None, None, e.clone(), s, s.clone())
    dw, db = (torch.full((24,), float("nan"), device="cuda") for _ in range(2))
    gpu_lib.layer_norm_bwd(e, e.clone(), None, s, s, e.clone(), dw, db)
    assert not dw.any() and not db.any()


def test_gradients_against_differences(gpu_lib):
    """<dx, v>, <dw, v>, <db, v> against central differences of
    L = sum dy * layer_norm(x) in float64 along random directions v: the
    difference quotient is off by h^2 |L'''| / 6, below 1e-7 of the
    derivative's scale here; the float32 gradients by the bounds above."""
    T, d, h = 6, 96, 1e-4
    x, dy, w, b = problem(12, T, d, outliers=False)
    mean, rstd = stats_of(x, 0.0)
    dx, dw, db = (torch.empty(s, device="cuda") for s in ((T, d), (d,), (d,)))
    gpu_lib.layer_norm_bwd(dy.cuda(), x.cuda(), w.cuda(), mean.cuda(), rstd.cuda(), dx, dw, db)
    loss = lambda x, w, b: float((dy.double() * ref_fwd(x, w, b, 0.0)[0]).sum())  # noqa: E731
    gen = torch.Generator().manual_seed(1)
    for k, grad in ((0, dx), (1, dw), (2, db)):
        for _ in range(4):
            args = [x.double(), w.double(), b.double()]
            v = torch.randn(args[k].shape, generator=gen).double()
            lo, hi = list(args), list(args)
            lo[k], hi[k] = args[k] - h * v, args[k] + h * v
            num = (loss(*hi) - loss(*lo)) / (2 * h)
            got = float((grad.double().cpu() * v).sum())
            scale = float(grad.double().cpu().norm() * v.norm())
            # mean and rstd enter the backward rounded to float32
            assert abs(num - got) <= 2e-6 * scale, (k, num, got, scale)


def test_repeats_other_stream_and_graph(gpu_lib):
    """The same bits on another stream, and in three replays of a captured
    graph with eager work between them."""
    T, d = 300, 1032
    x, dy, w, b = (t.cuda() for t in problem(20, T, d, BF16, F32))
    new = lambda: [torch.empty((T, d), dtype=BF16, device="cuda"), torch.empty(T, device="cuda"),  # noqa: E731
                   torch.empty(T, device="cuda"), torch.empty((T, d), device="cuda"),
                   torch.empty(d, device="cuda"), torch.empty(d, device="cuda")]
    ws = torch.empty(gpu_lib.layer_norm_bwd_workspace_bytes(T, d), dtype=torch.uint8,
                     device="cuda")

    def both(o, stream=None, w_=None):
        gpu_lib.layer_norm_fwd(x, w, b, o[0], o[1], o[2], stream=stream)
        gpu_lib.layer_norm_bwd(dy, x, w, o[1], o[2], o[3], o[4], o[5], ws=w_, stream=stream)

    ref = new()
    both(ref)
    torch.cuda.synchronize()
    side, on_side = torch.cuda.Stream(), new()
    both(on_side, stream=side)                      # the workspace belongs to that stream
    side.synchronize()
    assert all(torch.equal(a, r) for a, r in zip(on_side, ref))
    out = new()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(out, w_=ws)
    for _ in range(3):
        for t in out:
            t.fill_(float("nan"))
        x.mul_(2.0)
        graph.replay()
        torch.cuda.synchronize()
        again = new()
        both(again)
        torch.cuda.synchronize()
        assert all(torch.equal(a, r) for a, r in zip(out, again))
