"""LinearCrossEntropy as a layer: what it keeps between forward and backward."""
import pytest
import torch

pytestmark = pytest.mark.gpu

T, D, V = 130, 96, 500


def layer(fq, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    head = fq.LinearCrossEntropy(V, D, T)
    head.init_state(torch.empty((V, D), device="cuda").normal_(generator=g))
    x = torch.empty((T, D), device="cuda").normal_(generator=g)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[::5] = -1
    return head, x, target, torch.full((T,), 1 / T, device="cuda")


def test_the_target_may_be_overwritten_after_the_forward(gpu_lib):
    """As x may be: a loader that fills one buffer again before the backward."""
    head, x, target, dloss = layer(gpu_lib)
    head.forward(x, target)
    want = head.backward(dloss).clone()
    head.forward(x, target)
    target.random_(0, V)
    x.zero_()
    assert torch.equal(head.backward(dloss), want)
    head.forward(x, target)
    assert not torch.equal(head.backward(dloss), want)


@pytest.mark.parametrize("raw", [False, True])
def test_on_another_stream(gpu_lib, raw):
    """The copy is on the call's stream, behind what was sent to it before: a target that is
    still being written there."""
    head, x, target, dloss = layer(gpu_lib)
    head.forward(x, target)
    want = head.backward(dloss).clone()
    stream = torch.cuda.Stream()
    new, busy = torch.zeros_like(target), torch.zeros(1 << 26, device="cuda")
    torch.cuda.synchronize()
    arg = stream.cuda_stream if raw else stream
    with torch.cuda.stream(stream):
        for _ in range(20):
            busy.add_(1)
        new.copy_(target)
    head.forward(x, new, stream=arg)
    dx = head.backward(dloss, stream=arg)
    torch.cuda.synchronize()
    assert torch.equal(dx, want)


def test_a_graph_reads_the_target_that_is_there(gpu_lib):
    head, x, target, dloss = layer(gpu_lib)
    head.forward(x, target)
    want = head.backward(dloss).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        head.forward(x, target)
        head.backward(dloss)
    good = target.clone()
    for k in range(4):
        target.random_(0, V)
        graph.replay()
        torch.cuda.synchronize()
        assert not torch.equal(head.dx, want)
        target.copy_(good)
        head.dx.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(head.dx, want), k


def test_targets_are_checked_before_anything_runs(gpu_lib):
    head, x, target, dloss = layer(gpu_lib)
    head.forward(x, target)
    want = head.xq.clone()
    for bad in (target.int(), target[1:], target.cpu(), torch.stack((target, target), 1)[:, 0]):
        with pytest.raises(gpu_lib.FalqError):
            head.forward(x + 1, bad)
    assert torch.equal(head.xq, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab, d, tokens", [(50, 32, 0), (1, 16, 1), (1, 16, 40), (300, 16, 1)])
def test_smallest_layers(gpu_lib, vocab, d, tokens, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    head = gpu_lib.LinearCrossEntropy(vocab, d, tokens, dx_dtype=dtype)
    head.init_state(torch.empty((vocab, d), device="cuda").normal_(generator=g))
    x = torch.empty((tokens, d), device="cuda").normal_(generator=g)
    target = torch.zeros(tokens, dtype=torch.int64, device="cuda")
    loss = head.forward(x, target)
    dx = head.backward(torch.ones(tokens, device="cuda"))
    assert loss.shape == (tokens,) and dx.shape == (tokens, d)
    if vocab == 1:
        # dx = w expm1(z - lse) with lse = z: z is summed twice, once in float32 with 16 + 6
        # roundings of its absolute sum and its scale's 4 half steps, lse has k's three, the
        # two products' with k and ln 2 and ln 2's own, 2^-24 of z each
        dec = lambda q, s: q.view(torch.float8_e4m3fn).double() / s.double()  # noqa: E731
        terms = dec(head.xq, head.s_x) * dec(head.wq, head.s_w)
        off = (22 * terms.abs().sum(1) + 10 * terms.sum(1).abs()) * 2.0 ** -24
        most = off[:, None] * dec(head.wq, head.s_w).abs()
        assert not bool(loss.any()) and bool((dx.abs() <= most * (1 + 2.0 ** -7) + 1e-30).all())
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(dx).all())
