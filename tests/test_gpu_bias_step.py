"""A layer's bias is trained with its adapters: adapter_update steps it by its
clipped gradient, with SGD and with AdamW.

SGD: b - lr g with a rounding each (the GPU's float32 operations, so equal bits).
AdamW, per step and element: the moments, the quotient and the step take eight
roundings of terms no larger than those in `tol` below, and the scalars one each."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = torch.bfloat16
T, D, FF, R = 40, 48, 80, 4


def layer(fq, seed=0, **kw):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
    m = fq.MeldedLinear(FF, D, R, T, bias=True, act="silu", y_dtype=BF16, **kw)
    m.init_state(rn(FF, D), rn(R, D), rn(FF, R) * 1e-2, bias=rn(FF))
    return m, rn


def test_init_state_sets_the_bias(gpu_lib):
    m, _ = layer(gpu_lib)
    assert m.bias.abs().sum() > 0
    kept = m.bias.clone()
    m.init_state(torch.randn(FF, D).cuda(), m.A.clone(), m.B.clone())
    assert torch.equal(m.bias, kept)                        # not given: left as it is
    plain = gpu_lib.MeldedLinear(FF, D, R, T)
    with pytest.raises(ValueError):
        plain.init_state(torch.randn(FF, D).cuda(), torch.randn(R, D).cuda(),
                         torch.randn(FF, R).cuda(), bias=torch.zeros(FF).cuda())


def test_sgd(gpu_lib):
    m, rn = layer(gpu_lib)
    x, dy, res = rn(T, D), rn(T, FF), rn(T, FF).to(BF16)
    m.forward(x, residual=res)
    m.backward(dy)
    norm = torch.empty(1, device="cuda")
    gpu_lib.clip_gradients([m], 0.1, norm)
    before, g = m.bias.clone(), m.dbias.clone()
    assert g.any()
    m.adapter_update(0.25)
    assert torch.equal(m.bias, before - 0.25 * g)
    a, b = layer(gpu_lib)[0], layer(gpu_lib)[0]
    a.forward(x, residual=res)
    a.backward(dy)
    a.update(1e-2, 0.5)
    b.step(x, dy, lr=1e-2, tau=0.5, residual=res)           # the same as one call
    assert torch.equal(a.y, b.y) and torch.equal(a.bias, b.bias) and torch.equal(a.A, b.A)


def test_adamw(gpu_lib):
    hyper = {"beta1": 0.8, "beta2": 0.95, "eps": 1e-6, "weight_decay": 0.1}
    m, rn = layer(gpu_lib, optimizer="adamw", adamw=hyper)
    lr, p = 0.05, m.bias.double()
    mo, vo, tol = torch.zeros_like(p), torch.zeros_like(p), torch.zeros_like(p)
    for t in range(1, 5):
        m.dA.copy_(rn(R, D)), m.dB.copy_(rn(FF, R)), m.dbias.copy_(rn(FF))
        g = m.dbias.double()
        m.adapter_update(lr)
        b1, b2 = (float(torch.tensor(hyper[k])) for k in ("beta1", "beta2"))
        mo = b1 * mo + (1 - b1) * g
        vo = b2 * vo + (1 - b2) * g * g
        step = lr / (1 - b1 ** t)
        den = vo.sqrt() / (1 - b2 ** t) ** 0.5 + hyper["eps"]
        p = p - step * mo / den                             # the bias does not decay
        # moments: up to 4 roundings a step of terms below max |g| so far, times the step
        tol = tol + U * p.abs() + 16 * t * U * step * (mo.abs() + 3.0) / den
        assert bool(((m.bias.double() - p).abs() <= tol).all()), t
    assert int(m.adam_state[0]) == 4


def test_captured(gpu_lib):
    """Replays step the bias on, as eager steps do."""
    for opt in ("sgd", "adamw"):
        (e, rn), (c, _) = layer(gpu_lib, optimizer=opt), layer(gpu_lib, optimizer=opt)
        x, dy = rn(T, D), rn(T, FF)
        for m in (e, c):
            m.step(x, dy)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.step(x, dy)
        for _ in range(3):
            graph.replay()
            e.step(x, dy)
            torch.cuda.synchronize()
            assert torch.equal(e.bias, c.bias) and torch.equal(e.B, c.B), opt
