"""A training step as a user runs it with the operators of the microscaled formats and
the loss: the norm's input and the activation's pre-activation kept in 8 bits, an MLP of
two melded linears, the loss over an FP8 output layer, and the whole way back; the same
step captured in a graph, on another stream, and beside another one.

Every call is checked against its formula in float64 on the inputs it got, within rel-L2
1e-3 where a product on the matrix cores is involved, half a step of bfloat16 (2^-8)
where an output has that type and 1e-5 elsewhere."""
import math

import numpy as np
import pytest
import torch

from tests import mx_ref

pytestmark = pytest.mark.gpu

F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8
T, D, FF, R, VOCAB = 200, 288, 800, 8, 1111


def rel(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def dec(q, s):
    return q.view(torch.float8_e4m3fn).double() / s.double()


def kept(q, e):
    n = q.shape[1]
    v = mx_ref.decode(q.cpu().numpy(), e.cpu().numpy().astype(int) - 127, "fp8")
    assert v.shape[1] == n
    return torch.from_numpy(v).cuda()


def gelu(z):
    return z * 0.5 * torch.erfc(-z / math.sqrt(2))


def gelu_slope(z):
    return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


class Step:
    def __init__(self, fq, seed=3, scratch=None):
        self.fq = fq
        g = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
        self.up = fq.MeldedLinear(FF, D, R, T, bias=True, act="gelu", y_dtype=BF16, keep_z="fp8",
                                  z_scratch=scratch)
        self.down = fq.MeldedLinear(D, FF, R, T, bias=True, y_dtype=BF16, dy_dtype=BF16)
        self.head = fq.LinearCrossEntropy(VOCAB, D, T, dx_dtype=BF16)
        for m in (self.up, self.down):
            m.init_state(rn(m.d_out, m.d_in) * m.d_in ** -0.5, rn(R, m.d_in) * R ** -0.5,
                         rn(m.d_out, R) * 1e-2, bias=rn(m.d_out) * 0.1)
        self.W = rn(VOCAB, D) * D ** -0.5
        self.head.init_state(self.W)
        self.w, self.b = 1 + 0.1 * rn(D), 0.1 * rn(D)
        self.x = rn(T, D).to(BF16)
        self.target = torch.randint(0, VOCAB, (T,), generator=g).cuda()
        self.target[::7] = -100
        self.dloss = (self.target >= 0).float() / float((self.target >= 0).sum())
        new = lambda *s, t=F32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        self.h, self.mean, self.rstd = new(T, D, t=BF16), new(T), new(T)
        self.x_q, self.x_e = new(T, D, t=U8), new(*fq.checkpoint_scales_shape(T, D), t=U8)
        self.dx, self.dw, self.db = new(T, D), new(D), new(D)
        self.ws_ln = new(max(1, fq.layer_norm_bwd_workspace_bytes(T, D)), t=U8)

    def run(self, stream=None):
        fq, s = self.fq, stream
        fq.layer_norm_fwd(self.x, self.w, self.b, self.h, self.mean, self.rstd, stream=s)
        fq.checkpoint_save(self.x, self.x_q, self.x_e, stream=s)
        self.up.forward(self.h, stream=s)
        self.down.forward(self.up.y, stream=s, residual=self.x)
        self.head.forward(self.down.y, self.target, stream=s)
        self.head.backward(self.dloss, stream=s)
        self.down.backward(self.head.dx, stream=s)
        self.up.backward(self.down.dx, stream=s)
        fq.layer_norm_bwd_ckpt(self.up.dx, self.x_q, self.x_e, self.w, self.mean, self.rstd,
                               self.dx, self.dw, self.db, ws=self.ws_ln, stream=s)

    def results(self):
        return [t.clone() for t in (self.head.loss, self.head.lse, self.head.dx, self.down.dx,
                                    self.up.dz, self.up.dx, self.up.dA, self.up.dB, self.up.dbias,
                                    self.down.dA, self.dx, self.dw, self.db, self.up.z_q,
                                    self.up.z_e)]


def same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


def test_every_call_of_a_step(gpu_lib):
    s = Step(gpu_lib)
    s.run()
    torch.cuda.synchronize()
    up, down, head = s.up, s.down, s.head
    xh, wh = dec(head.xq, head.s_x), dec(head.wq, head.s_w)
    z = xh @ wh.T
    keep = s.target >= 0
    at = s.target.clamp(min=0)[:, None]
    lse = torch.logsumexp(z, 1)
    loss = torch.where(keep, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    assert rel(head.lse, lse) <= 1e-5 and rel(head.loss, loss) <= 1e-5
    p = torch.exp(z - lse[:, None]).scatter_add_(1, at, -torch.ones_like(z[:, :1]))
    assert rel(head.dx, (p * s.dloss.double()[:, None]) @ wh) <= 2.0 ** -8
    assert not bool(head.dx[~keep].any())
    # down's gradient flows from it, up's through the pre-activation that 8 bits kept
    g2 = dec(down.gq, down.s_g)
    assert rel(down.dx, g2 @ dec(down.wq, down.s_w)) <= 1e-3
    zk = kept(up.z_q, up.z_e)
    zx = dec(up.xq, up.s_x) @ dec(up.wq, up.s_w).T + up.bias.double()
    # a code is off by half a step, 2^-4 of itself, or of the smallest normal one, 2^-10 of it
    amax = torch.nn.functional.pad(zx.abs(), (0, -FF % 32)).view(T, -1, 32).amax(2)
    amax = amax.repeat_interleave(32, 1)[:, :FF]
    assert bool(((zk - zx).abs() <= zx.abs() * (2.0 ** -4 + 2.0 ** -7) + amax * 2.0 ** -13).all())
    dz = down.dx.double() * gelu_slope(zk)
    assert rel(up.dz, dz) <= 1e-5 and rel(up.dbias, dz.sum(0)) <= 1e-5
    # the norm
    xk = kept(s.x_q, s.x_e)
    dh, xn = up.dx.double(), (xk - s.mean.double()[:, None]) * s.rstd.double()[:, None]
    g = dh * s.w.double()
    dx = s.rstd.double()[:, None] * (g - g.mean(1, keepdim=True)
                                     - xn * (g * xn).mean(1, keepdim=True))
    assert rel(s.dx, dx) <= 1e-5
    assert rel(s.dw, (dh * xn).sum(0)) <= 1e-5 and rel(s.db, dh.sum(0)) <= 1e-5


def test_the_gradients_that_8_bits_give_are_near_the_exact_ones(gpu_lib):
    """Against the same step with everything kept exactly: a pre-activation off by 2^-4
    of itself moves gelu's slope by at most 2^-4 |z| |gelu''(z)| <= 2^-4 0.49 (|z gelu''| has
    its largest value 0.485 at |z| = 0.83), beside slopes of 0.5 at the root mean square of 0.68: 4.5 % if
    every element were off by all of it."""
    a = Step(gpu_lib)
    a.run()
    exact, dz = torch.empty_like(a.up.dz), a.up.dz.clone()
    gpu_lib.linear_act_bwd(a.down.dx, a.up.z, exact, act="gelu")
    assert 0 < rel(dz, exact.double()) <= 0.045


def test_layers_share_the_scratch_of_z(gpu_lib):
    """Two steps whose layers share it, one after the other, as with one each."""
    scratch = torch.empty(T * FF + 5, dtype=BF16, device="cuda")
    a, b = Step(gpu_lib, 3, scratch), Step(gpu_lib, 4, scratch)
    c, d = Step(gpu_lib, 3), Step(gpu_lib, 4)
    for s in (a, b, c, d):
        s.fq.layer_norm_fwd(s.x, s.w, s.b, s.h, s.mean, s.rstd)
        s.up.forward(s.h)
    for s in (a, b, c, d):
        s.up.backward(s.up.y.float())
    for u, v in ((a, c), (b, d)):
        assert torch.equal(u.up.dz, v.up.dz) and torch.equal(u.up.dA, v.up.dA)


def test_a_captured_step_replays(gpu_lib):
    s = Step(gpu_lib)
    s.run()
    want = s.results()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        s.run()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    other = Step(gpu_lib, 9)
    for k in range(4):
        for t in (s.head.loss, s.head.dx, s.dx, s.up.dz, s.dw):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(s.results(), want), k
        other.run()                                # eager work between the replays
        torch.cuda.synchronize()
    # new inputs in the same places
    x0, x1 = s.x.clone(), (s.x * 0.5 + 0.25)
    s.x.copy_(x1)
    s.target.copy_(s.target.flip(0))
    s.dloss.copy_((s.target >= 0).float() / float((s.target >= 0).sum()))
    graph.replay()
    torch.cuda.synchronize()
    got = s.results()
    s.run()
    assert same(got, s.results()) and not same(got, want) and not torch.equal(x0, s.x)


def test_another_stream_and_two_at_once(gpu_lib):
    steps = [Step(gpu_lib, k) for k in (5, 6)]
    want = []
    for s in steps:
        s.run()
        want.append(s.results())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        for s in steps:
            s.dx.zero_()
            s.head.loss.zero_()
        torch.cuda.synchronize()
        for s, st in zip(steps, streams):          # by the stream argument, no torch context
            s.run(stream=st)
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            assert same(s.results(), w)


def test_workspaces_of_the_calls_own(gpu_lib):
    """Without `ws` each call takes its own, on the stream it runs on."""
    fq, s = gpu_lib, Step(gpu_lib, 7)
    s.run()
    st = torch.cuda.Stream()
    h = s.head
    torch.cuda.synchronize()
    loss, lse, dx = torch.empty_like(h.loss), torch.empty_like(h.lse), torch.empty_like(h.dx)
    fq.linear_cross_entropy_fwd(h.xq, h.s_x, h.wq, h.s_w, s.target, loss, lse, stream=st)
    fq.linear_cross_entropy_bwd(h.xq, h.s_x, h.wq, h.s_w, s.target, lse, s.dloss, dx, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(loss, h.loss) and torch.equal(lse, h.lse) and torch.equal(dx, h.dx)


def test_the_model_in_fp4(gpu_lib):
    """The same MLP evaluated with FP4 operands, and its loss: products against the
    formula on the operands' values."""
    fq, s = gpu_lib, Step(gpu_lib)
    s.run()
    g = torch.Generator().manual_seed(11)
    wu, wd = torch.randn(FF, D, generator=g).cuda() * D ** -0.5, torch.randn(
        D, FF, generator=g).cuda() * FF ** -0.5

    def operand(x):
        q = torch.empty((x.shape[0], x.shape[1] // 2), dtype=U8, device="cuda")
        e = torch.empty(fq.mxfp4_scales_shape(*x.shape), dtype=U8, device="cuda")
        fq.mxfp4_quantize(x, q, e)
        v = torch.empty(x.shape, device="cuda")
        fq.mxfp4_dequantize(q, e, v)
        return (q, e), v.double()
    (up, vu), (down, vd) = operand(wu), operand(wd)
    (h, vh) = operand(s.h)
    y1, y2 = torch.empty((T, FF), dtype=BF16, device="cuda"), s.x.clone()
    fq.melded_linear_fwd_mxfp4(*h, *up, y1, bias=s.up.bias, act="gelu")
    assert rel(y1, gelu(vh @ vu.T + s.up.bias.double())) <= 2.0 ** -8
    a, va = operand(y1)
    fq.melded_linear_fwd_mxfp4(*a, *down, y2, bias=s.down.bias, residual=y2)
    assert rel(y2, va @ vd.T + s.down.bias.double() + s.x.double()) <= 2.0 ** -8
    loss = s.head.forward(y2, s.target)
    z = dec(s.head.xq, s.head.s_x) @ dec(s.head.wq, s.head.s_w).T
    want = torch.nn.functional.cross_entropy(z, s.target, ignore_index=-100, reduction="none")
    assert rel(loss, want) <= 1e-5
    assert np.isfinite(float(loss.sum()))
