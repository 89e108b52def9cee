"""grad_norm / grad_clip on the GPU against the formula in float64.

Tolerances (u = 2^-24): squares are summed in float64, so the norm is the
exact one rounded once (u, and a float64 sum's error far below it).  The call
takes max_norm as float32 (one rounding of the float64 the reference divides),
the coefficient is rounded once and the product once, so a clipped element is
off by three roundings, (1 + u)^3 - 1 < 3.1 u, plus, for bfloat16, half a step
of its type."""
import math

import pytest
import torch

from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def make(sizes, dtypes, seed=0, std=1e-2, views=True):
    """Tensors as views at any element of one buffer per type, or on their own."""
    g = torch.Generator().manual_seed(seed)
    out, at, buf = [], {F32: 3, BF16: 5}, {}
    for t in (F32, BF16):
        n = sum(s for s, dt in zip(sizes, dtypes) if dt == t) + 64
        buf[t] = (torch.randn(n, generator=g) * std).to(t).cuda()
    for n, t in zip(sizes, dtypes):
        v = buf[t][at[t]: at[t] + n]
        at[t] += n
        out.append(v if views else v.clone())
    return out


def norm_ref(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def check(grads, before, norm, max_norm, eps):
    ref = norm_ref(before)
    assert abs(float(norm) - ref) <= 1.001 * U * ref
    coef = min(1.0, max_norm / (ref + eps))
    for g, b in zip(grads, before):
        want = b.double() * coef
        tol = want.abs() * (3.1 * U + (2.0 ** -8 if g.dtype == BF16 and coef < 1 else 0)) + 1e-37
        assert bool(((g.double() - want).abs() <= tol).all())


CASES = [
    ([1], [F32]), ([0], [F32]), ([0, 5, 0], [F32, BF16, BF16]), ([7, 8, 9, 8191, 8192, 8193],
                                                                 [F32] * 6),
    ([64 * 4096, 4096 * 64], [F32, F32]), ([1000003], [BF16]),
    ([3 + 37 * i for i in range(130)], [(F32, BF16)[i % 3 == 1] for i in range(130)]),
    ([1 + (i * 7919) % 5000 for i in range(448)], [F32] * 448),
    ([20_000_011, 5], [F32, BF16]), ([2, 3, 1, 4, 5, 6, 7, 15, 16, 17], [BF16] * 10),
    ([1, 2, 3, 4, 5, 1023, 1024, 1025, 2047, 2049, 4097], [F32, BF16] * 5 + [F32]),
]


@pytest.mark.parametrize("views", [True, False])
@pytest.mark.parametrize("sizes,dtypes", CASES)
def test_norm_and_clip(gpu_lib, sizes, dtypes, views):
    announce(f"grad_clip {len(sizes)} tensors, {sum(sizes)} elements, views={views}")
    grads = make(sizes, dtypes, len(sizes), views=views)
    before = [g.clone() for g in grads]
    ref = norm_ref(before)
    norm = torch.full((1,), float("nan"), device="cuda")
    gpu_lib.grad_norm(grads, norm)
    assert abs(float(norm) - ref) <= 1.001 * U * ref
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    # clipped, into other tensors (aligned otherwise than the inputs) and in place
    out = [torch.full((g.numel() + 1,), float("nan"), dtype=g.dtype, device="cuda")[1:]
           for g in grads]
    for max_norm in (0.5 * ref, 2.0 * ref + 1.0, math.inf, 0.0):
        norm.fill_(float("nan"))
        gpu_lib.grad_clip(grads, max_norm, norm, out=out)
        check(out, before, norm, max_norm, 1e-6)
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
    gpu_lib.grad_clip(grads, 2.0 * ref + 1.0, norm)        # not clipped: left as they are
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    if ref > 0:                                            # eps = 0 on a norm of 0 is 0 / 0
        gpu_lib.grad_clip(grads, 0.25 * ref, norm, eps=0.0)
        check(grads, before, norm, 0.25 * ref, 0.0)


def test_neighbours_are_left_alone(gpu_lib):
    """Views inside a buffer: nothing before, between or behind them changes."""
    buf = torch.arange(1.0, 40001.0, device="cuda")
    keep = buf.clone()
    grads = [buf[1:8], buf[11:9000], buf[9001:39990]]
    norm = torch.empty(1, device="cuda")
    gpu_lib.grad_clip(grads, 1.0, norm)
    inside = torch.zeros(40000, dtype=torch.bool, device="cuda")
    for a, b in ((1, 8), (11, 9000), (9001, 39990)):
        inside[a:b] = True
    assert torch.equal(buf[~inside], keep[~inside]) and (buf[inside] < keep[inside]).all()


def test_nothing_and_not_finite(gpu_lib):
    norm = torch.full((1,), float("nan"), device="cuda")
    gpu_lib.grad_norm([], norm)
    assert float(norm) == 0.0
    norm.fill_(float("nan"))
    gpu_lib.grad_clip([], 1.0, norm)
    assert float(norm) == 0.0
    for bad in (float("nan"), float("inf")):
        g = [torch.ones(100, device="cuda"), torch.ones(9, device="cuda", dtype=BF16)]
        g[0][50] = bad
        gpu_lib.grad_clip(g, 1.0, norm)
        if math.isnan(bad):
            assert math.isnan(float(norm)) and torch.isnan(g[0]).all() and torch.isnan(g[1]).all()
        else:
            assert math.isinf(float(norm)) and torch.isnan(g[0][50]) and not g[1].any()
    # squares beyond float32's range
    g = [torch.full((1000,), 1e30, device="cuda"), torch.full((1000,), 1e-30, device="cuda")]
    gpu_lib.grad_norm(g, norm)
    assert abs(float(norm) / (1e30 * math.sqrt(1000.0)) - 1) <= 3 * U
    gpu_lib.grad_norm(g[1:], norm)
    assert abs(float(norm) / (1e-30 * math.sqrt(1000.0)) - 1) <= 3 * U


def test_overlaps_are_refused(gpu_lib):
    g = torch.ones(1000, device="cuda")
    norm = torch.empty(1, device="cuda")
    o = torch.empty(1000, device="cuda")
    for grads, out in (([g, g], None), ([g[:600], g[599:]], None), ([g[:500], g[500:]], [o[:500],
                       o[499:999]]), ([g[:500], g[500:]], [g[500:], o[:500]]),
                       ([g[:500]], [g[1:501]])):
        with pytest.raises(gpu_lib.FalqError):
            gpu_lib.grad_clip(grads, 1.0, norm, out=out)
    gpu_lib.grad_norm([g, g], norm)                        # the norm alone may count one twice
    assert abs(float(norm) - math.sqrt(2000.0)) <= U * 45
    gpu_lib.grad_clip([g[:500], g[500:]], 1.0, norm, out=[g[:500], o[:500]])
    assert abs(float(norm) - math.sqrt(1000.0)) <= U * 32


def test_repeats_other_stream_and_graph(gpu_lib):
    """The same bits on another stream, and in three replays of a captured
    graph with eager work between them."""
    grads = make([100_003, 5, 70_000, 1_000_001], [F32, BF16, BF16, F32], 3)
    out = [torch.empty_like(g) for g in grads]
    norm = torch.empty(1, device="cuda")
    gpu_lib.grad_clip(grads, 1.0, norm, out=out)
    torch.cuda.synchronize()
    want, wn = [o.clone() for o in out], norm.clone()
    side = torch.cuda.Stream()
    for o in out:
        o.zero_()
    torch.cuda.synchronize()
    gpu_lib.grad_clip(grads, 1.0, norm, out=out, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(norm, wn)
    ws = torch.empty(gpu_lib.grad_norm_workspace_bytes(4), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.grad_clip(grads, 1.0, norm, out=out, ws=ws)
    for k in range(3):
        for g in grads:
            g.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        got, gn = [o.clone() for o in out], norm.clone()
        gpu_lib.grad_clip(grads, 1.0, norm, out=out)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, got)) and torch.equal(norm, gn)
