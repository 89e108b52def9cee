"""A training step of two melded linears with the operators around them, as a
block uses them: layer norm, quantize, product with bias and gelu, quantize,
product with bias and residual; the backward of each; the gradients of both
layers, the biases and the norm clipped by their global norm; the adapter step.

Every call is checked against its formula in float64 on the inputs it got (the
FP8 codes are taken from the GPU: rounding to them is a step function), within
rel-L2 1e-3 where a product on the matrix cores is involved, half a step of
bfloat16 (2^-8) where an output has that type and 1e-5 elsewhere (sums of a few
hundred float32 terms)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
T, D, FF, R = 200, 272, 784, 8
LR, EPS = 1e-2, 1e-6


def rel(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def dec(q, s):
    return q.view(torch.float8_e4m3fn).double() / s.double()


class Block:
    def __init__(self, fq, y_dtype):
        self.fq = fq
        g = torch.Generator().manual_seed(3)
        rn = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
        self.up = fq.MeldedLinear(FF, D, R, T, bias=True, act="gelu", y_dtype=BF16)
        self.down = fq.MeldedLinear(D, FF, R, T, bias=True, y_dtype=y_dtype, dy_dtype=y_dtype)
        for m in (self.up, self.down):
            m.init_state(rn(m.d_out, m.d_in) * m.d_in ** -0.5, rn(R, m.d_in) * R ** -0.5,
                         rn(m.d_out, R) * 1e-2)
            m.bias.copy_(rn(m.d_out) * 0.1)
        self.w, self.b = 1 + 0.1 * rn(D), 0.1 * rn(D)
        self.x, self.dy = rn(T, D).to(y_dtype), (rn(T, D) * 1e-2).to(y_dtype)
        self.h = torch.empty((T, D), dtype=BF16, device="cuda")
        self.mean, self.rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        self.dw, self.db = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
        self.dx = torch.empty((T, D), device="cuda")
        self.norm = torch.empty(1, device="cuda")
        self.ws_ln = torch.empty(max(1, fq.layer_norm_bwd_workspace_bytes(T, D)),
                                 dtype=torch.uint8, device="cuda")
        self.ws_clip = torch.empty(fq.grad_norm_workspace_bytes(8), dtype=torch.uint8,
                                   device="cuda")

    def grads(self):
        return [*(t for m in (self.up, self.down) for t in (m.dA, m.dB, m.dbias)), self.dw,
                self.db]

    def forward_backward(self):
        fq = self.fq
        fq.layer_norm_fwd(self.x, self.w, self.b, self.h, self.mean, self.rstd)
        self.up.forward(self.h)
        self.down.forward(self.up.y, residual=self.x)
        self.down.backward(self.dy)
        self.up.backward(self.down.dx)
        fq.layer_norm_bwd(self.up.dx, self.x, self.w, self.mean, self.rstd, self.dx, self.dw,
                          self.db, ws=self.ws_ln)

    def clip_and_step(self, max_norm):
        self.fq.clip_gradients([self.up, self.down], max_norm, self.norm,
                               extra=[self.dw, self.db], eps=EPS, ws=self.ws_clip)
        for m in (self.up, self.down):
            m.adapter_update(LR)

    def step(self, max_norm):
        self.forward_backward()
        self.clip_and_step(max_norm)


def gelu(z):
    return z * 0.5 * torch.erfc(-z / math.sqrt(2))


def gelu_slope(z):
    return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


@pytest.mark.parametrize("y_dtype", [torch.float32, BF16])
def test_block_step(gpu_lib, y_dtype):
    blk = Block(gpu_lib, y_dtype)
    up, down = blk.up, blk.down
    tol_y = 2.0 ** -8 if y_dtype == BF16 else 1e-3
    blk.forward_backward()
    torch.cuda.synchronize()
    # forward
    x = blk.x.double()
    mu = x.mean(1, keepdim=True)
    rstd = ((x - mu).square().mean(1, keepdim=True) + 1e-5) ** -0.5
    assert rel(blk.h, (x - mu) * rstd * blk.w.double() + blk.b.double()) <= 2.0 ** -8
    xq, wq = dec(up.xq, up.s_x), dec(up.wq, up.s_w)
    z = xq @ wq.T + up.bias.double()
    assert rel(up.z, z) <= 2.0 ** -8 and rel(up.y, gelu(z)) <= 2.0 ** -8
    xq2, wq2 = dec(down.xq, down.s_x), dec(down.wq, down.s_w)
    assert rel(down.y, xq2 @ wq2.T + down.bias.double() + x) <= tol_y
    # backward of the down projection (its upstream gradient is dy itself)
    assert down.dz is None
    assert rel(down.dbias, blk.dy.double().sum(0)) <= 1e-5
    g2 = dec(down.gq, down.s_g)
    assert rel(down.dx, g2 @ wq2) <= 1e-3
    assert rel(down.dA, (g2 @ down.B.double()).T @ xq2) <= 1e-3
    assert rel(down.dB, g2.T @ (xq2 @ down.A.double().T)) <= 1e-3
    # through the activation and the up projection
    dz = down.dx.double() * gelu_slope(up.z.double())
    assert rel(up.dz, dz) <= 1e-5 and rel(up.dbias, dz.sum(0)) <= 1e-5
    g1 = dec(up.gq, up.s_g)
    assert rel(up.dx, g1 @ wq) <= 1e-3
    assert rel(up.dA, (g1 @ up.B.double()).T @ xq) <= 1e-3
    assert rel(up.dB, g1.T @ (xq @ up.A.double().T)) <= 1e-3
    # the norm
    dh, xh = up.dx.double(), (x - blk.mean.double()[:, None]) * blk.rstd.double()[:, None]
    g = dh * blk.w.double()
    dx = blk.rstd.double()[:, None] * (g - g.mean(1, keepdim=True)
                                       - xh * (g * xh).mean(1, keepdim=True))
    assert rel(blk.dx, dx) <= 1e-5
    assert rel(blk.dw, (dh * xh).sum(0)) <= 1e-5 and rel(blk.db, dh.sum(0)) <= 1e-5
    # clipping, and the adapter step on the clipped gradients
    before = [t.clone() for t in blk.grads()]
    adapters = [t.clone() for m in (up, down) for t in (m.A, m.B)]
    norm = math.sqrt(sum(float(t.double().square().sum()) for t in before))
    blk.clip_and_step(0.5 * norm)
    assert abs(float(blk.norm) / norm - 1) <= 2.0 ** -23
    coef = 0.5 * norm / (norm + EPS)
    for t, b in zip(blk.grads(), before):
        assert rel(t, b.double() * coef) <= 2.0 ** -22
    clipped = [t for m in (up, down) for t in (m.dA, m.dB)]
    for t, b, gr in zip([t for m in (up, down) for t in (m.A, m.B)], adapters, clipped):
        assert rel(t, b.double() - LR * gr.double()) <= 2.0 ** -23


def test_block_step_captured(gpu_lib):
    """Steps replayed from a captured graph, eager work between them, against
    the same steps run eagerly: the same bits."""
    eager, graphed = Block(gpu_lib, torch.float32), Block(gpu_lib, torch.float32)
    graphed.step(0.05)                                     # once before the capture, as eager
    eager.step(0.05)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        graphed.step(0.05)
    for k in range(3):
        for blk in (eager, graphed):
            blk.x.mul_(1.125)
            blk.dy.add_(1e-3)
        graph.replay()
        torch.cuda.synchronize()
        eager.step(0.05)
        torch.cuda.synchronize()
        for a, b in zip([*eager.grads(), eager.dx, eager.down.y, eager.norm, eager.up.A,
                         eager.down.B],
                        [*graphed.grads(), graphed.dx, graphed.down.y, graphed.norm, graphed.up.A,
                         graphed.down.B]):
            assert torch.equal(a, b), k


def test_layers_with_an_epilogue(gpu_lib):
    """What a layer refuses, and that one without bias or activation but with a
    bf16 output takes dY straight."""
    fq = gpu_lib
    with pytest.raises(ValueError):
        fq.MeldedLinear(64, 32, 4, 16, act="tanh")
    with pytest.raises(ValueError):
        fq.MeldedLinear(64, 32, 4, 16, bias=True, fp8_a=True)
    with pytest.raises(ValueError):
        fq.MeldedLinear(64, 32, 4, 16, y_dtype=torch.float16)
    plain = fq.MeldedLinear(64, 32, 4, 16)
    plain.init_state(torch.randn(64, 32).cuda(), torch.randn(4, 32).cuda(),
                     torch.randn(64, 4).cuda())
    with pytest.raises(ValueError):
        plain.forward(torch.randn(16, 32).cuda(), residual=torch.zeros(16, 64).cuda())
    m = fq.MeldedLinear(64, 32, 4, 16, y_dtype=BF16)
    m.init_state(torch.randn(64, 32).cuda(), torch.randn(4, 32).cuda(),
                 torch.randn(64, 4).cuda())
    x, dy = torch.randn(16, 32).cuda(), torch.randn(16, 64).cuda()
    m.forward(x)
    assert rel(m.y, dec(m.xq, m.s_x) @ dec(m.wq, m.s_w).T) <= 2.0 ** -8
    m.backward(dy)
    assert rel(m.dx, dec(m.gq, m.s_g) @ dec(m.wq, m.s_w)) <= 1e-3 and m.dz is None
    m.step(x, dy)


@pytest.mark.parametrize("T, D", [(1, 16), (5, 48), (300, 272)])
def test_tensors_side_by_side(gpu_lib, T, D):
    """All tensors of a call carved from one buffer without gaps: nothing is
    refused, and every output is what separate tensors give."""
    fq, dev = gpu_lib, "cuda"
    f32 = torch.float32
    rows, vec, col = (f32, (T, D)), (f32, (D,)), (f32, (T,))
    one = (f32, (1,))

    def carved(*kinds):
        need = sum(torch.empty(s, dtype=t).numel() * t.itemsize for t, s in kinds)
        buf, at, out = torch.zeros(need, dtype=torch.uint8, device=dev), 0, []
        for t, s in kinds:
            k = math.prod(s) * t.itemsize
            out.append(buf[at:at + k].view(t).view(s))
            at += k
        return out

    def apart(*kinds):
        return [torch.zeros(s, dtype=t, device=dev) for t, s in kinds]

    g = torch.Generator().manual_seed(5)
    draw = lambda s: torch.randn(s, generator=g).cuda()  # noqa: E731
    X, DY, W, B, RES = draw((T, D)), draw((T, D)), draw(D), draw(D), draw((T, D))
    Xq, sx = torch.empty((T, D), dtype=torch.uint8, device=dev), torch.empty(1, device=dev)
    fq.fp8_quantize(X, Xq, sx)
    Wq, sw = torch.empty((D, D), dtype=torch.uint8, device=dev), torch.empty(1, device=dev)
    fq.fp8_quantize(draw((D, D)), Wq, sw)
    got = []
    for place in (carved, apart):
        x, y, dy, w, b, dw, db, mean, rstd = place(rows, rows, rows, vec, vec, vec, vec, col, col)
        x.copy_(X), dy.copy_(DY), w.copy_(W), b.copy_(B)
        fq.layer_norm_fwd(x, w, b, y, mean, rstd)
        fq.layer_norm_bwd(dy, x, w, mean, rstd, dy, dw, db)
        xq, wq, res, o, z, bias, s1, s2 = place((torch.uint8, (T, D)), (torch.uint8, (D, D)), rows,
                                                rows, rows, vec, one, one)
        xq.copy_(Xq), wq.copy_(Wq), res.copy_(RES), bias.copy_(B), s1.copy_(sx), s2.copy_(sw)
        fq.melded_linear_fwd_act(xq, s1, wq, s2, o, bias=bias, act="gelu", residual=res, z=z)
        d2, z2, dbias = place(rows, rows, vec)
        d2.copy_(DY), z2.copy_(z)
        fq.linear_act_bwd(d2, z2, d2, dbias=dbias, act="gelu")
        g0, g1, o0, o1, norm = place(rows, vec, rows, vec, one)
        g0.copy_(d2), g1.copy_(dbias)
        fq.grad_clip([g0, g1], 0.5, norm, out=[o0, o1])
        got.append((y, mean, rstd, dy, dw, db, o, z, d2, dbias, o0, o1, norm, x, w, xq, res, g0))
    for i, (a, b) in enumerate(zip(*got)):
        assert torch.equal(a, b), i
