"""Sums over the rows of tensors of more than 2^31 elements, exact: every summand is
1, -1 or 0, so each sum is an integer below 2^24, which float32 holds in whatever
order it is formed, and one row too many or too few shows."""
import pytest
import torch

from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
SHAPES = [(270_000, 8192), (270_011, 8191), (70_001, 32_768), (1_100_003, 2048), (2_200_000, 977)]


@pytest.fixture(scope="module", params=SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def signs(request):
    """Two matrices of random signs."""
    T, D = request.param
    announce(f"{T} x {D}")
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    out = []
    for _ in range(2):
        t = torch.empty((T, D), dtype=BF16, device="cuda")
        t.random_(0, 2, generator=g)
        out.append(t.mul_(2).sub_(1))
    assert out[0].numel() > 2 ** 31
    yield out
    del out, t
    torch.cuda.empty_cache()


def column_sums(f, *t):
    out = torch.zeros(t[0].shape[1], dtype=torch.float64, device="cuda")
    step = max(1, 2 ** 26 // t[0].shape[1])
    for a in range(0, t[0].shape[0], step):
        out += f(*(x[a:a + step] for x in t)).to(F32).sum(0).double()
    return out


def test_layer_norm(gpu_lib, signs):
    """mean 0 and rstd 1: dweight = sum dy x, dbias = sum dy."""
    dy, x = signs
    T, D = x.shape
    dw, db = (torch.full((D,), float("nan"), device="cuda") for _ in range(2))
    gpu_lib.layer_norm_bwd(dy, x, None, torch.zeros(T, device="cuda"), torch.ones(T, device="cuda"),
                           None, dw, db)
    assert torch.equal(db.double(), column_sums(lambda g: g, dy))
    assert torch.equal(dw.double(), column_sums(lambda g, v: g * v, dy, x))


@pytest.mark.parametrize("act", ["none", "relu"])
def test_activation(gpu_lib, signs, act):
    dy, z = signs
    db = torch.full((z.shape[1],), float("nan"), device="cuda")
    gpu_lib.linear_act_bwd(dy, None if act == "none" else z, None, dbias=db, act=act)
    ref = (column_sums(lambda g: g, dy) if act == "none"
           else column_sums(lambda g, v: g * (v > 0), dy, z))
    assert torch.equal(db.double(), ref)
