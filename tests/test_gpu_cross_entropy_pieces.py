"""linear_cross_entropy_bwd over three and more pieces of the vocabulary, whose sums a middle
piece reads and writes back, by whole tiles and by splits, into either type; and over
strips of rows with several pieces each, the last of them with a width, splits and a
workspace's layout of its own.  Sampled rows against the definition in float64."""
import pytest
import torch

from tests.gpu_util import announce
from tests.loss_mx_plan import loss as plan
from tests.test_gpu_cross_entropy import Case, within
from tests.test_gpu_cross_entropy_float32 import reference

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16

# (T, d, V): dx's kernel and the pieces of a whole strip, and of the last one
SHAPES = [
    ((16384, 48, 70000), ("64*", 5), ("64*", 5)),
    ((12000, 272, 70001), ("128*", 4), ("128*", 4)),
    ((16384, 1040, 50000), ("128", 4), ("128", 4)),
    ((9000, 2064, 90000), ("256x128*", 4), ("256x128*", 4)),
    ((16384, 2064, 50000), ("256x128", 4), ("256x128", 4)),
    ((16384, 4096, 50000), ("256", 4), ("256", 4)),
    ((16400, 48, 40000), ("64*", 3), ("32x64*", 1)),
    ((17084, 272, 50001), ("256x128", 4), ("64*", 1)),
    ((25384, 48, 70000), ("64*", 5), ("64*", 3)),
    ((32771, 16, 33000), ("64*", 3), ("32x64*", 1)),
]


class Rows:
    """Some rows of a case, for its references."""

    def __init__(self, c, rows):
        self.T, self.d, self.V, self.wv, self.wm = len(rows), c.d, c.V, c.wv, c.wm
        self.xv, self.xm = c.xv[rows], c.xm[rows]
        self.target, self.dloss = c.target[rows], c.dloss[rows]
        self.reference = lambda lse: Case.reference(self, lse)


@pytest.mark.parametrize("shape, whole, last", SHAPES)
def test_sampled_rows(gpu_lib, shape, whole, last):
    announce(f"pieces, T, d, V = {shape}")
    T, d, V = shape
    assert plan(*shape)[2: 4] == whole and plan((T - 1) % 16384 + 1, d, V)[2: 4] == last
    c = Case(*shape)
    loss, lse = c.forward(gpu_lib)
    # the ends of the strips, and some between
    at = sorted({r for a in range(0, T, 16384) for b in (min(T, a + 16384),)
                 for r in (a, a + 1, (a + b) // 2, b - 2, b - 1)} & set(range(T)))
    rows = torch.tensor(at, device="cuda")
    # a target in each piece, the first and the last class
    some = torch.linspace(0, V - 1, len(at), device="cuda").long()
    c.target[rows[:-1]] = some[:-1]
    c.target[rows[-1]] = V - 1
    loss, lse = c.forward(gpu_lib)
    part = Rows(c, rows)
    r = part.reference(lse[rows])
    within(lse[rows], r[1], r[4], "lse")
    within(loss[rows], r[0], r[3], "loss")
    dx = c.backward(gpu_lib, lse, BF16)
    within(dx[rows], r[2], r[5], "dx")
    assert bool(torch.isfinite(dx).all()) and not bool(dx[c.target < 0].any())
    dx = c.backward(gpu_lib, lse, F32)
    within(dx[rows], *reference(part, lse[rows]), "float32 dx")
    assert bool(torch.isfinite(dx).all()) and not bool(dx[c.target < 0].any())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_workspace_for_all_strips(gpu_lib, dtype):
    """Each strip's rows as a call of their own gives them, bit for bit, in a workspace of
    exactly the size asked for that was full of NaN, and nothing behind it is written."""
    T, d, V = 16384 + 700, 272, 50001
    c = Case(T, d, V)
    loss, lse = c.forward(gpu_lib)
    n = gpu_lib.linear_cross_entropy_bwd_workspace_bytes(T, d, V, dtype)
    ws = torch.full((n + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    dx = torch.full((T, d), float("nan"), dtype=dtype, device="cuda")
    gpu_lib.linear_cross_entropy_bwd(*c.args, lse, c.dloss, dx, ws=ws[:n])
    assert bool((ws[n:] == 0xFF).all())
    for a in (0, 16384):
        s = slice(a, min(T, a + 16384))
        one = torch.empty((s.stop - s.start, d), dtype=dtype, device="cuda")
        gpu_lib.linear_cross_entropy_bwd(c.xq[s], c.s_x, c.wq, c.s_w, c.target[s], lse[s],
                                         c.dloss[s], one)
        assert torch.equal(dx[s], one)
