"""linear_cross_entropy_fwd and linear_cross_entropy_bwd where a logit is a small sum of large
terms: two codes of each eight cancel, and what is left of the other six is a ten
thousandth of them."""
import pytest
import torch

from tests.gpu_util import announce
from tests.loss_mx_plan import loss as plan

pytestmark = pytest.mark.gpu

F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8

# every kernel of G
SHAPES = {
    "32x64": [(1, 16, 2), (64, 16, 3), (50, 48, 70)],
    "64": [(5000, 272, 77)],
    "128": [(2100, 512, 9001)],
    "192x128": [(3000, 3088, 3001)],
    "256x128": [(2048, 2064, 3001)],
    "256": [(4096, 4096, 8000)],
}
CASES = [(k, s) for k, v in SHAPES.items() for s in v]


class Case:
    """Logits of a standard deviation of `spread`."""

    def __init__(self, T, d, V, spread=4.0, big=448.0, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + T + d + V)

        def rows(n, second):
            v = torch.empty((n, d // 8, 8), device="cuda").normal_(generator=g) * 4
            v[:, :, 0] = big
            v[:, :, 1] = second * big
            return v.view(n, d).to(torch.float8_e4m3fn)
        x, w = rows(T, 1.0), rows(V, -1.0)
        self.T, self.d, self.V = T, d, V
        self.s_x = torch.full((1,), 16 * (d * 6 / 8) ** 0.5 / spread, device="cuda")
        self.s_w = torch.ones(1, device="cuda")
        self.xv, self.wv = x.double() / self.s_x.double(), w.double()
        self.target = torch.randint(0, V, (T,), generator=g, device="cuda")
        self.dloss = torch.empty(T, device="cuda").normal_(generator=g) * 1e-2
        self.args = (x.view(U8), self.s_x, w.view(U8), self.s_w, self.target)

    def forward(self, fq):
        loss, lse = torch.full((2, self.T), float("nan"), device="cuda")
        fq.linear_cross_entropy_fwd(*self.args, loss, lse)
        return loss, lse

    def backward(self, fq, lse, dtype):
        dx = torch.full((self.T, self.d), float("nan"), dtype=dtype, device="cuda")
        fq.linear_cross_entropy_bwd(*self.args, lse, self.dloss, dx)
        return dx


@pytest.mark.parametrize("kind, shape", CASES)
def test_probabilities_are_one_at_most(gpu_lib, kind, shape):
    """Whatever a logit's error, dx is a sum of V terms of at most |dloss| |w| each."""
    announce(f"cancelling terms, T, d, V = {shape}")
    assert plan(*shape)[1] == kind
    c = Case(*shape)
    loss, lse = c.forward(gpu_lib)
    assert float(lse.abs().max()) < 100
    # (the terms' half steps, and that of the sum in dx's type)
    most = c.dloss.abs().double()[:, None] * c.wv.abs().sum(0) * (1 + 2.0 ** -7)
    for dt in (F32, BF16):
        assert bool((c.backward(gpu_lib, lse, dt).abs() <= most).all())


@pytest.mark.parametrize("size", [1e5, 1e7, 1e8])
@pytest.mark.parametrize("T, d, V", [(64, 16, 3), (300, 272, 999)])
def test_a_target_does_not_pass_lse(gpu_lib, T, d, V, size):
    """Logits whose half steps are units: the target's own logit, summed apart, may lie above
    lse, and its probability is 1 at most all the same."""
    announce(f"logits of {size}, T, d, V = {(T, d, V)}")
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = torch.empty((T, d), device="cuda").normal_(generator=g).to(torch.float8_e4m3fn)
    w = torch.empty((V, d), device="cuda").normal_(generator=g).to(torch.float8_e4m3fn)
    s_x, s_w = torch.full((2, 1), (d ** 0.5 / size) ** 0.5, device="cuda")
    target = (x.double() @ w.double().T).argmax(1)
    args = (x.view(U8), s_x, w.view(U8), s_w, target)
    loss, lse = torch.empty((2, T), device="cuda")
    gpu_lib.linear_cross_entropy_fwd(*args, loss, lse)
    assert bool(torch.isfinite(lse).all())
    most = w.double().abs().sum(0) / s_w.double() * (1 + 2.0 ** -7)
    for dt in (F32, BF16):
        dx = torch.empty((T, d), dtype=dt, device="cuda")
        gpu_lib.linear_cross_entropy_bwd(*args, lse, torch.ones(T, device="cuda"), dx)
        assert bool((dx.abs() <= most).all())


@pytest.mark.parametrize("size", [1.0, 100.0, 1e4, 1e6, 1e9, 1e11])
@pytest.mark.parametrize("T, d, V", [(64, 16, 3), (300, 272, 999), (700, 1040, 5001)])
def test_a_sure_token_has_no_loss(gpu_lib, T, d, V, size):
    """The target's logit is the largest, in exact sums of whole numbers: loss = log of the
    sum of exp(differences), each difference off by four half steps (k's two roundings, the
    difference's product with it, the exponential's own), 2^-21 of it with a factor of two to
    spare; the sum and its logarithm by 2^-20 of one and of the loss.  Never below 0.  And
    lse is finite at any size of a logit, and off by as much of itself besides."""
    announce(f"sure tokens at logits of {size}, T, d, V = {(T, d, V)}")
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    # whole numbers up to 8: every sum of d products is exact
    x = torch.randint(-8, 9, (T, d), generator=g, device="cuda").float()
    w = torch.randint(-8, 9, (V, d), generator=g, device="cuda").float()
    s_x, s_w = torch.full((2, 1), (25 * d ** 0.5 / size) ** 0.5, device="cuda")
    f8 = lambda t: t.to(torch.float8_e4m3fn).view(U8)  # noqa: E731
    sums = x.double() @ w.double().T
    target = sums.argmax(1)
    loss, lse = torch.empty((2, T), device="cuda")
    gpu_lib.linear_cross_entropy_fwd(f8(x), s_x, f8(w), s_w, target, loss, lse)
    # k is rounded a few times, as are the differences' products with it
    z = sums / (s_x.double() * s_w.double())
    diff = z - z.gather(1, target[:, None])
    want = torch.log(torch.exp(diff).sum(1))
    grown = torch.exp(diff) * diff.abs() * 2.0 ** -21            # an exponential's error
    tol = grown.sum(1) / torch.exp(want) + (want + 1) * 2.0 ** -20
    assert bool(((loss - want).abs() <= tol).all())
    assert bool((loss >= 0).all())
    ref = torch.logsumexp(z, 1)
    assert bool(((lse - ref).abs() <= tol + ref.abs() * 2.0 ** -21).all())


def powers(v):
    """The largest power of two in each eight of a row of codes."""
    e = torch.where(v == 0, -6.0, v.abs().clamp(min=2.0 ** -6).log2().floor())
    return torch.exp2(e.view(v.shape[0], -1, 8).amax(2))


def bf16_reference(c, lse):
    """dx and its tolerance (u = 2^-24) where FP8's logits are off by e, 7 2^-13 of the largest
    product's power of two of each eight, (d / 8 + 2) u of the absolute sum and 8 u |z|: p lies
    between p exp(-e) and the smaller of p exp(e) and 1, whatever e is; the rest as in
    tests/test_gpu_cross_entropy.py."""
    u = 2.0 ** -24
    w = c.wv
    z, S = c.xv @ w.T, c.xv.abs() @ w.abs().T
    s = c.s_x.double()
    e = (powers(c.xv * s) / s) @ powers(w).T * (7 * 2.0 ** -13) + S * ((c.d / 8 + 2) * u)
    given = lse.double()[:, None]
    e += 8 * u * z.abs() + 2 * u * given.abs() + 2.0 ** -20
    p = torch.exp((z - given).clamp(max=0))      # (lse itself is off by what its sums are)
    onehot = torch.zeros_like(p).scatter_(1, c.target[:, None], 1.0)
    G = p - onehot
    et = S * ((16 * -(-c.d // 1024) + 6) * u + (c.d / 4 + 8) * u) + 4 * u * (z.abs() + given.abs())
    EG = torch.maximum(p * -torch.expm1(-e), torch.exp((z - given + e).clamp(max=0)) - p)
    EGt = torch.maximum(p * -torch.expm1(-et), torch.exp((z - given + et).clamp(max=0)) - p)
    EG = torch.where(onehot > 0, EGt + 2.0 ** -20 * G.abs(), EG)
    EG += (G.abs() + EG) * 2.0 ** -11 + 2.0 ** -40
    f = c.dloss.double()[:, None]
    dx = f * (G @ w)
    tol = f.abs() * (EG @ w.abs() + (G.abs() @ w.abs()) * ((c.V / 4 + 8) * u)) + 4 * u * dx.abs()
    return dx, tol + (dx.abs() + tol) * 2.0 ** -8 + 1e-37


@pytest.mark.parametrize("spread", [0.5, 4.0, 100.0])
@pytest.mark.parametrize("big", [8.0, 64.0, 448.0])
@pytest.mark.parametrize("shape", [(64, 16, 3), (50, 48, 70), (5000, 272, 77), (2100, 512, 9001)])
def test_bfloat16_is_off_by_its_logits_error(gpu_lib, shape, big, spread):
    announce(f"bfloat16 gradient of cancelling terms, T, d, V = {shape}, {big}, {spread}")
    c = Case(*shape, spread=spread, big=big)
    loss, lse = c.forward(gpu_lib)
    dx = c.backward(gpu_lib, lse, BF16)
    ref, tol = bf16_reference(c, lse)
    assert bool(((dx.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [2, 3, 64, 1000])
def test_classes_alike_and_lse_near_zero(gpu_lib, V, dtype):
    """All rows of the weight the same, with terms that cancel: every p is 1 / V to what half a
    step of lse makes of it (lse is 0 up to its rounding, as the logits are -log V), though
    FP8's logits are alike as well; so dx = dloss w (V / V - 1) = 0, up to the terms' errors,
    2^-11 of each in bfloat16, and their sums'."""
    d, T = 32, 40
    w = torch.zeros(d, device="cuda")
    w[0], w[1], w[2:8] = 448, -448, 1
    x = torch.zeros(d, device="cuda")
    x[0], x[1], x[2:8] = 448, 448, -1
    f8 = lambda t, n: t.to(torch.float8_e4m3fn).view(U8).repeat(n, 1)  # noqa: E731
    s = torch.full((1,), 6 / float(torch.log(torch.tensor(float(V)))), device="cuda")
    one = torch.ones(1, device="cuda")
    target = torch.arange(T, device="cuda") % V
    args = (f8(x, T), s, f8(w, V), one, target)
    loss, lse = torch.empty((2, T), device="cuda")
    gpu_lib.linear_cross_entropy_fwd(*args, loss, lse)
    assert float(lse.abs().max()) <= 1e-5
    assert float((loss - 6 / float(s)).abs().max()) <= 1e-5
    dx = torch.empty((T, d), dtype=dtype, device="cuda")
    gpu_lib.linear_cross_entropy_bwd(*args, lse, torch.ones(T, device="cuda"), dx)
    # of the logit -6 / s = -log V, FP8 may drop all six ones (each 2^-17 of 448^2)
    off = 1e-5 if dtype == F32 else float(torch.expm1(6 / s))
    tol = (off + 2.0 ** -10 + (V / 4 + 8) * 2.0 ** -24) * w.abs() * 2
    assert bool((dx.abs() <= tol * (1 + 2.0 ** -7) + 1e-30).all())
