"""linear_cross_entropy_fwd and linear_cross_entropy_bwd against their definition in
float64, every element, for each of their kernels, and the gradient against differences
of the loss.

Tolerances (u = 2^-24).  Forward: the codes are multiplied as float16, exactly, and
summed in float32: a logit is off by (d / 4 + 8) u sum |x w| / s + 4 u |z|, lse by at
most the largest of a row's logits' errors, and besides by its own evaluation: the
exponents' rounding (their arguments are formed by one fused step, and what counts lies
within 2^5 of the maximum: 2^6 u), the exponential's and logarithm's 4 u, sums of up to 64
+ runs terms, and 2 u |lse|.
Backward: G's logits are FP8's (tests/gpu_util.gemm_bound), so p is off by expm1 of
their error and lse's rounding, besides 2^-20 of itself; the target's logit is summed
in float32: a lane adds 16 products of each 1024 codes, one rounding each, and the
wave's sum is six more, (16 ceil(d / 1024) + 6) u of the absolute sum, and 4 u of itself;
G is rounded to float16, whose half step is 2^-11 of a number with eleven bits (1 + 2^-11
lies between two of them), below 2^-29 by 2^-40 absolutely; their products with the
weight are summed in float32, (V / 4 + 8) u of the absolute sum; the row's factor 4 u;
then half a step of dx's type."""
import math

import pytest
import torch

from tests.gpu_util import announce
from tests.loss_mx_plan import loss as plan

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8

# (T, d, V): every kernel of the forward, of G and of dx; rows, columns and K steps that
# end inside a tile, one piece of the vocabulary and several, strips of rows
SHAPES = {
    ("64", "32x64", "32x64", 1): [(1, 16, 700), (17, 48, 77), (129, 16, 65), (300, 64, 999)],
    ("64", "32x64", "32x64*", 1): [(16, 272, 3001), (40, 64, 5000)],
    ("32x64", "32x64", "32x64*", 1): [(7, 4112, 2000), (16, 4112, 5000)],
    ("64", "64", "32x64*", 1): [(100, 272, 9000)],
    ("64", "64", "64", 1): [(5000, 272, 77)],
    ("32x64", "32x64", "64", 1): [(700, 4096, 700), (1024, 2064, 63), (1100, 4112, 129)],
    ("64", "64", "128", 1): [(3000, 2064, 129)],
    ("128", "128", "256x128*", 1): [(1024, 1040, 20001)],
    ("128", "128", "128*", 1): [(2100, 512, 9001)],
    ("128", "256x128", "64", 1): [(5000, 272, 3001)],
    ("128", "256x128", "128*", 1): [(600, 528, 20000)],
    ("128", "256x128", "128", 1): [(2048, 1040, 12000)],
    ("128", "192x128", "128", 1): [(3000, 3088, 3001)],
    ("128", "256x128", "256x128", 1): [(2048, 2064, 3001)],
    ("256", "256", "256", 1): [(4096, 4096, 8000)],
    ("128", "192x128", "64*", 1): [(2100, 48, 40000)],
    ("256", "192x128", "128*", 1): [(513, 1040, 20000)],
    ("256", "256x128", "128*", 1): [(4096, 1040, 20001)],
    ("128", "128", "64*", 2): [(9000, 48, 40000)],
    ("128", "192x128", "256x128*", 2): [(9000, 272, 33000)],
    ("256", "256", "256x128", 2): [(10000, 2064, 28000)],
    ("256", "256", "128*", 1): [(4100, 2064, 14001)],
}


def codes(x):
    s = (448.0 / x.abs().max()).reshape(1)
    q = (x * s).clamp(-448, 448).to(torch.float8_e4m3fn)
    v = q.double()
    e = torch.where(v == 0, -6.0, v.abs().clamp(min=2.0 ** -6).log2().floor())
    return q.view(U8), s, v / s.double(), torch.exp2(e.view(x.shape[0], -1, 8).amax(2)) / s.double()


class Case:
    def __init__(self, T, d, V, gain=1.5, seed=0, ignored=0.2):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + T + d + V)
        rn = lambda *s: torch.empty(s, device="cuda").normal_(generator=g)  # noqa: E731
        x = rn(T, d) * torch.exp(gain * torch.rand((T, 1), generator=g, device="cuda"))
        x[:, ::100] *= 10
        self.T, self.d, self.V = T, d, V
        self.xq, self.s_x, self.xv, self.xm = codes(x)
        self.wq, self.s_w, self.wv, self.wm = codes(rn(V, d) * (gain / math.sqrt(d)))
        t = torch.randint(0, V, (T,), generator=g, device="cuda")
        gone = torch.rand(T, generator=g, device="cuda") < ignored
        self.target = torch.where(gone, torch.full_like(t, -100), t)
        self.dloss = rn(T) * 1e-2
        self.args = (self.xq, self.s_x, self.wq, self.s_w, self.target)

    def forward(self, fq, **k):
        loss, lse = torch.full((2, self.T), float("nan"), device="cuda")
        fq.linear_cross_entropy_fwd(*self.args, loss, lse, **k)
        return loss, lse

    def backward(self, fq, lse, dtype, **k):
        dx = torch.full((self.T, self.d), float("nan"), dtype=dtype, device="cuda")
        fq.linear_cross_entropy_bwd(*self.args, lse, self.dloss, dx, **k)
        return dx

    def reference(self, lse=None):
        """loss, lse, dx and their tolerances; lse: the one that the backward was given"""
        z = self.xv @ self.wv.T
        S = self.xv.abs() @ self.wv.abs().T
        ez = S * ((self.d / 4 + 8) * U) + 4 * U * z.abs()
        ref_lse = torch.logsumexp(z, 1)
        runs = self.V / 16
        e_lse = ez.amax(1) + (64 + 4 + 64 + runs) * U + 2 * U * ref_lse.abs()
        keep = self.target >= 0
        at = self.target.clamp(min=0)[:, None]
        zt = z.gather(1, at)[:, 0]
        loss = torch.where(keep, ref_lse - zt, torch.zeros_like(zt))
        e_loss = torch.where(keep, e_lse + ez.gather(1, at)[:, 0] + 4 * U * loss.abs(),
                             torch.zeros_like(zt))
        given = ref_lse if lse is None else lse.double()
        p = torch.exp(z - given[:, None])
        onehot = torch.zeros_like(p).scatter_(1, at, 1.0)
        G = p - onehot
        e8 = (self.xm @ self.wm.T) * (7 * 2.0 ** -13) + S * ((self.d / 8 + 2) * U) + 8 * U * z.abs()
        EG = p * torch.expm1(e8 + 2 * U * given.abs()[:, None] + 2.0 ** -20)
        et = (S * ((16 * -(-self.d // 1024) + 6) * U) + 4 * U * z.abs() + 2 * U * given.abs()[:, None])
        EG = torch.where(onehot > 0, p * torch.expm1(et) + 2.0 ** -20 * G.abs(), EG)
        EG += (G.abs() + EG) * 2.0 ** -11 + 2.0 ** -40
        aw = self.wv.abs()
        f = torch.where(keep, self.dloss.double(), torch.zeros_like(zt))[:, None]
        dx = f * (G @ self.wv)
        tol = f.abs() * (EG @ aw + (G.abs() @ aw) * ((self.V / 4 + 8) * U)) + 4 * U * dx.abs()
        return loss, ref_lse, dx, e_loss, e_lse, tol


def within(got, ref, tol, name):
    tol = tol + (ref.abs() + tol) * (torch.finfo(got.dtype).eps / 2) + 1e-37
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (f"{name}: {int(bad.sum())} of {bad.numel()}, the first at "
                                 f"{bad.nonzero()[0].tolist()}, worst "
                                 f"{float((err / tol).nan_to_num(nan=math.inf).max()):.3g}")


def check(fq, c, dtypes=(F32, BF16)):
    loss, lse = c.forward(fq)
    r = c.reference(lse)
    within(lse, r[1], r[4], "lse")
    within(loss, r[0], r[3], "loss")
    assert bool((loss[c.target < 0] == 0).all())
    for dt in dtypes:
        dx = c.backward(fq, lse, dt)
        within(dx, r[2], r[5], f"dx {dt}")
        assert not bool(dx[c.target < 0].any())


CASES = [(k, s) for k, v in SHAPES.items() for s in v]


@pytest.mark.parametrize("kinds, shape", CASES)
def test_every_kernel(gpu_lib, kinds, shape):
    announce(f"linear_cross_entropy T, d, V = {shape}")
    got = plan(*shape)
    assert got[:4] == kinds and got[4] == 1, got
    check(gpu_lib, Case(*shape))


def test_strips_of_rows(gpu_lib):
    """More rows than a strip, the last strip of few tokens, or of more of them."""
    for T in (16384 + 5, 2 * 16384 + 100):
        announce(f"linear_cross_entropy T = {T}")
        assert plan(T, 16, 100)[4] > 1
        check(gpu_lib, Case(T, 16, 100))


@pytest.mark.parametrize("T", [1, 20, 200])
@pytest.mark.parametrize("V", [1, 2, 63, 64, 65])
def test_small_vocabularies(gpu_lib, T, V):
    c = Case(T, 32, V)
    check(gpu_lib, c)
    if V == 1:                                      # the only class: no loss, no gradient
        loss, lse = c.forward(gpu_lib)
        assert float(loss.abs().max()) <= 1e-5
        assert float(c.backward(gpu_lib, lse, F32).abs().max()) <= 1e-6


def test_sure_and_flat_tokens(gpu_lib):
    """Logits of hundreds, where all but one exponential underflow, and zeros."""
    c = Case(70, 64, 1500, ignored=0.0)
    c.s_x, c.xv, c.xm = c.s_x / 40, c.xv * 40, c.xm * 40
    c.args = (c.xq, c.s_x, c.wq, c.s_w, c.target)
    check(gpu_lib, c)
    z = c.xv @ c.wv.T
    assert float((z.amax(1) - z.amin(1)).max()) > 200
    c.target.copy_(z.argmax(1))                     # right and sure: small losses, not 0 - 0
    check(gpu_lib, c)
    c.xq.zero_()
    c.xv, c.xm = c.xv * 0, c.xm * 0 + 2.0 ** -6 / float(c.s_x)
    loss, lse = c.forward(gpu_lib)
    assert float((lse.double() - math.log(1500)).abs().max()) <= 1e-5
    check(gpu_lib, c)


@pytest.mark.parametrize("T,d,V", [(5, 64, 500), (70, 528, 2000), (700, 1040, 3001)])
def test_logits_of_tens_of_thousands(gpu_lib, T, d, V):
    """The FP8 product's logits are then off by more than one, and pass lse: what they give
    is bounded, a sure token's gradient 0 up to the others' terms."""
    c = Case(T, d, V, ignored=0.0)
    c.s_x.copy_(c.s_x / 2e4)
    z = c.xv @ c.wv.T * 2e4
    c.target.copy_(z.argmax(1))
    loss, lse = c.forward(gpu_lib)
    assert bool(((lse - z.amax(1)).abs() <= z.amax(1) * 1e-4 + 1).all())
    for dt in (F32, BF16):
        dx = c.backward(gpu_lib, lse, dt)
        # each of V terms at most |dloss| |w|, half a step of dx's type aside
        most = c.dloss.abs()[:, None].double() * c.wv.abs().sum(0)
        assert bool((dx.abs() <= most * (1 + 2.0 ** -7) + 1e-30).all())


@pytest.mark.parametrize("T,d,V", [(16, 272, 9282), (40, 528, 41389), (100, 528, 8620),
                                   (333, 16, 20536), (700, 48, 26825)])
def test_splits_left_without_columns(gpu_lib, T, d, V):
    """Of dx's splits the last ones begin past the vocabulary."""
    check(gpu_lib, Case(T, d, V))


@pytest.mark.parametrize("T", [3, 50, 700])
def test_targets_out_of_range_and_nan(gpu_lib, T):
    """All tokens without a class; a class of V or more and a NaN in a row give NaN in
    that row only."""
    c = Case(T, 64, 333, ignored=0.0)
    c.target.fill_(-1)
    loss, lse = c.forward(gpu_lib)
    assert not bool(loss.any()) and bool(torch.isfinite(lse).all())
    assert not bool(c.backward(gpu_lib, lse, F32).any())
    c.target.fill_(5)
    c.target[1] = 333
    c.target[2] = 1 << 40
    c.xq[0, 7] = 0x7F                               # NaN
    for dt in (F32, BF16):
        loss, lse = c.forward(gpu_lib)
        dx = c.backward(gpu_lib, lse, dt)
        assert bool(loss[:3].isnan().all()) and bool(torch.isfinite(loss[3:]).all())
        assert bool(dx[:3].isnan().all()) and bool(torch.isfinite(dx[3:].float()).all())
    c.target[0] = -7                                # a NaN in a row that does not count
    loss, lse = c.forward(gpu_lib)
    assert float(loss[0]) == 0 and not bool(c.backward(gpu_lib, lse, F32)[0].any())


@pytest.mark.parametrize("T,d,V", [(3, 16, 65), (3, 16, 64), (50, 64, 129), (700, 64, 1025),
                                   (1, 4112, 2049)])
def test_nan_logits_reach_lse(gpu_lib, T, d, V):
    """A NaN in a row of the weight is in every token's sum, though it stand alone in the
    last run of columns; all logits of a token NaN give a NaN, not the empty sum's -inf."""
    c = Case(T, d, V, ignored=0.0)
    c.target.fill_(0)
    w = c.wq.clone()
    c.wq[-1, 3] = 0x7F
    loss, lse = c.forward(gpu_lib)
    assert bool(lse.isnan().all()) and bool(loss.isnan().all())
    assert bool(c.backward(gpu_lib, lse, F32).isnan().all())
    c.wq.copy_(w)
    c.xq[T // 2, 5] = 0xFF
    c.target[T // 2] = -1
    loss, lse = c.forward(gpu_lib)
    assert lse.isnan().nonzero().tolist() == [[T // 2]] and not bool(loss.isnan().any())


def test_gradient_against_differences(gpu_lib):
    """Central differences of the float64 loss along random directions, in the values
    that the codes stand for."""
    c = Case(40, 48, 600)
    loss, lse = c.forward(gpu_lib)
    dx = c.backward(gpu_lib, lse, F32).double()
    keep = c.target >= 0
    at = c.target.clamp(min=0)[:, None]

    def total(x):
        z = x @ c.wv.T
        each = torch.logsumexp(z, 1) - z.gather(1, at)[:, 0]
        return float((each * c.dloss.double())[keep].sum())
    # the differences' own error: h^2 / 6 of the third derivative, at most (2 max |v w|)^3 of
    # the weights, and float64's rounding over h
    h = 1e-4
    for seed in range(6):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        v = torch.empty(c.xv.shape, dtype=torch.float64, device="cuda").normal_(generator=g)
        diff = (total(c.xv + h * v) - total(c.xv - h * v)) / (2 * h)
        tol = float((c.reference(lse)[5] * v.abs()).sum())
        third = (2 * (v @ c.wv.T).abs().amax(1)) ** 3 * c.dloss.double().abs()
        tol += h * h / 6 * float(third.sum()) + 1e-15 * 40 * 10 / h
        tol += float((dx * v).abs().sum()) * U
        assert abs(diff - float((dx * v).sum())) <= tol


def test_results_repeat(gpu_lib):
    for shape in ((9, 256, 5000), (300, 272, 9000), (1024, 1040, 20001)):
        c = Case(*shape)
        loss, lse = c.forward(gpu_lib)
        dx = c.backward(gpu_lib, lse, F32)
        for _ in range(3):
            a, b = c.forward(gpu_lib)
            assert torch.equal(a, loss) and torch.equal(b, lse)
            assert torch.equal(c.backward(gpu_lib, lse, F32), dx)


def test_lse_may_be_left_out_and_nothing_else_is_written(gpu_lib):
    c = Case(33, 64, 500)
    loss, lse = c.forward(gpu_lib)
    buf = torch.full((33 + 16,), 7.0, device="cuda")
    gpu_lib.linear_cross_entropy_fwd(*c.args, buf[8: 41])
    assert torch.equal(buf[8: 41], loss)
    assert bool((buf[:8] == 7).all()) and bool((buf[41:] == 7).all())
    out = torch.full((35, 64), 7.0, dtype=BF16, device="cuda")
    gpu_lib.linear_cross_entropy_bwd(*c.args, lse, c.dloss, out[1: 34])
    assert torch.equal(out[1: 34], c.backward(gpu_lib, lse, BF16))
    assert bool((out[0] == 7).all()) and bool((out[34] == 7).all())


def test_no_tokens(gpu_lib):
    c = Case(4, 32, 50)
    none = lambda *s, t=F32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    gpu_lib.linear_cross_entropy_fwd(none(0, 32, t=U8), c.s_x, c.wq, c.s_w,
                                     none(0, t=torch.int64), none(0), none(0))
    gpu_lib.linear_cross_entropy_bwd(none(0, 32, t=U8), c.s_x, c.wq, c.s_w,
                                     none(0, t=torch.int64), none(0), none(0), none(0, 32))
