"""Tensors whose offsets pass 32 bits: the microscaled formats' calls, the FP4 product and
the cross entropy at rows past 2^31 and 2^32 elements or bytes, against the same calls on
those rows alone, or their definition in float64."""
import math

import pytest
import torch

from tests.loss_mx_plan import mx as plan

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8
D, T = 32768 + 32, 140000                                   # 4.6e9 elements


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def new(*s, t=U8):
    return torch.empty(s, dtype=t, device="cuda")


def filled(rows, d, t=BF16):
    """Rows that differ: a random one, shifted by the row's number and scaled by it."""
    base = torch.empty(2 * d, device="cuda")
    base.normal_(generator=torch.Generator("cuda").manual_seed(5))
    x = new(rows, d, t=t)
    for a in range(0, rows, 4096):
        n = min(4096, rows - a)
        i = torch.arange(a, a + n, device="cuda")
        at = (i * 977 % d)[:, None] + torch.arange(d, device="cuda")
        x[a: a + n] = base[at] * (1 + i[:, None] % 13)
    return x


def parts(rows):
    """Ranges of rows around 2^31 and 2^32 elements and at the end (multiples of 16 first)."""
    for at in (2 ** 31 // D // 16 * 16 - 16, 2 ** 32 // D // 16 * 16 - 16, (rows - 40) // 16 * 16):
        yield at, min(40, rows - at)


def test_checkpoints(gpu_lib):
    x = filled(T, D)
    q, e = new(T, D), new(*gpu_lib.checkpoint_scales_shape(T, D))
    gpu_lib.checkpoint_save(x, q, e)
    back = new(T, D, t=BF16)
    gpu_lib.checkpoint_restore(q, e, back)
    dz = new(T, D, t=BF16)
    gpu_lib.linear_act_bwd_ckpt(x, q, e, dz, act="relu")
    w, mean, rstd = new(D, t=F32).normal_(), new(T, t=F32).normal_(), new(T, t=F32).uniform_(0.5, 2)
    dx = new(T, D, t=BF16)
    gpu_lib.layer_norm_bwd_ckpt(x, q, e, w, mean, rstd, dx)
    for at, n in parts(T):
        s = slice(at, at + n)
        qs, es = new(n, D), new(*gpu_lib.checkpoint_scales_shape(n, D))
        gpu_lib.checkpoint_save(x[s], qs, es)
        assert torch.equal(q[s], qs) and torch.equal(e[s], es)
        a, b, c = new(n, D, t=BF16), new(n, D, t=BF16), new(n, D, t=BF16)
        gpu_lib.checkpoint_restore(qs, es, a)
        gpu_lib.linear_act_bwd_ckpt(x[s], qs, es, b, act="relu")
        gpu_lib.layer_norm_bwd_ckpt(x[s], qs, es, w, mean[s], rstd[s], c)
        assert torch.equal(back[s], a) and torch.equal(dz[s], b) and torch.equal(dx[s], c)
        # (a code is off by at most a 16th; the smallest normal one of a block is 2^-14 of
        # its largest)
        assert float((a.float() - x[s].float()).abs().max()) <= float(x[s].abs().max()) / 16


def test_fp4_operands(gpu_lib):
    x = filled(T, D)
    q, e = new(T, D // 2), new(*gpu_lib.mxfp4_scales_shape(T, D))
    gpu_lib.mxfp4_quantize(x, q, e)
    back = new(T, D, t=BF16)
    gpu_lib.mxfp4_dequantize(q, e, back)
    for at, n in parts(T):
        s = slice(at, at + n)
        qs, es = new(n, D // 2), new(*gpu_lib.mxfp4_scales_shape(n, D))
        gpu_lib.mxfp4_quantize(x[s], qs, es)
        assert torch.equal(q[s], qs) and torch.equal(e[:, s], es[:, :n])
        a = new(n, D, t=BF16)
        gpu_lib.mxfp4_dequantize(qs, es, a)
        assert torch.equal(back[s], a)


@pytest.mark.parametrize("tokens", [5, 29, 70, 300])
def test_fp4_product_of_a_far_weight(gpu_lib, tokens):
    """4.7e9 bytes of weight: the last columns as those rows' own product gives them."""
    d_in, d_out = 65536 + 32, 143376
    wq = torch.randint(0, 256, (d_out, d_in // 2), dtype=U8, device="cuda")
    w_e = torch.randint(120, 130, gpu_lib.mxfp4_scales_shape(d_out, d_in), dtype=U8, device="cuda")
    x = filled(tokens, d_in)
    xq, x_e = new(tokens, d_in // 2), new(*gpu_lib.mxfp4_scales_shape(tokens, d_in))
    gpu_lib.mxfp4_quantize(x, xq, x_e)
    y = new(tokens, d_out, t=F32)
    gpu_lib.melded_linear_fwd_mxfp4(xq, x_e, wq, w_e, y)
    xv = new(tokens, d_in, t=F32)
    gpu_lib.mxfp4_dequantize(xq, x_e, xv)
    for at in (2 ** 31 // (d_in // 2) // 16 * 16 - 16, 2 ** 32 // (d_in // 2) // 16 * 16 - 16,
               d_out - 48):
        wv = new(48, d_in, t=F32)
        gpu_lib.mxfp4_dequantize(wq[at: at + 48].contiguous(), w_e[:, at: at + 48].contiguous(), wv)
        ref, S = xv.double() @ wv.double().T, xv.abs().double() @ wv.abs().double().T
        # float32 sums of d_in products, and what a matrix instruction may drop of them
        assert bool(((y[:, at: at + 48] - ref).abs() <= S * (d_in / 4 + 8) * 2.0 ** -24).all())


def test_cross_entropy_of_a_far_weight(gpu_lib):
    """2.7e9 codes of weight, targets at its end and before and behind 2^31."""
    V, d, n = 131071, 20480, 6
    wq = new(V, d)
    for a in range(0, V, 8192):
        wq[a: a + 8192] = (torch.empty((min(8192, V - a), d), device="cuda").normal_() * 64
                           ).to(torch.float8_e4m3fn).view(U8)
    x = torch.empty((n, d), device="cuda").normal_().to(torch.float8_e4m3fn)
    s_x, s_w = torch.tensor([1.0], device="cuda"), torch.tensor([64 * math.sqrt(d)], device="cuda")
    edge = 2 ** 31 // d
    target = torch.tensor([V - 1, edge, edge + 1, 0, -1, V - 2], device="cuda")
    loss, lse = new(n, t=F32), new(n, t=F32)
    gpu_lib.linear_cross_entropy_fwd(x.view(U8), s_x, wq, s_w, target, loss, lse)
    dloss = torch.ones(n, device="cuda")
    dx = new(n, d, t=F32)
    gpu_lib.linear_cross_entropy_bwd(x.view(U8), s_x, wq, s_w, target, lse, dloss, dx)
    k = 1 / float(s_w)
    W = [wq[a: a + 8192].view(torch.float8_e4m3fn) for a in range(0, V, 8192)]
    z = torch.cat([x.double() @ w.double().T * k for w in W], 1)
    ref = torch.logsumexp(z, 1)
    keep = target >= 0
    at = target.clamp(min=0)[:, None]
    ref_loss = torch.where(keep, ref - z.gather(1, at)[:, 0], torch.zeros_like(ref))
    # float32 sums of d products, whose absolute sum is about 0.64 sqrt(d)
    tol = (d / 4 + 8) * 2.0 ** -24 * math.sqrt(d) + 1e-5
    assert float((lse - ref).abs().max()) <= tol and float((loss - ref_loss).abs().max()) <= 2 * tol
    G = torch.exp(z - ref[:, None])
    G.scatter_(1, at, G.gather(1, at) - 1)
    G[~keep] = 0
    want = sum(G[:, a: a + 8192] @ w.double() for a, w in zip(range(0, V, 8192), W)) * k
    # FP8's products of d codes are off by 2^-13 of the largest of each eight
    assert float((dx - want).norm()) <= 2e-3 * float(want.norm())
    assert not bool(dx[4].any())


@pytest.mark.parametrize("tokens,d_out,kind", [(66000, 33008, "256x128"), (8192, 11008, "128"),
                                               (8190, 16400, "128")])
def test_fp4_product_of_far_outputs(gpu_lib, tokens, d_out, kind):
    """2.2e9 outputs, and outputs that go past the caches in either kind of tile; 64
    products each, so that float32's sums are off by 64 half steps of their absolute sum
    at most."""
    d_in = 64
    assert plan(tokens, d_in, d_out) == kind
    x, w = filled(tokens, d_in), filled(d_out, d_in)
    ops = []
    for t in (x, w):
        q, e = new(len(t), d_in // 2), new(*gpu_lib.mxfp4_scales_shape(len(t), d_in))
        gpu_lib.mxfp4_quantize(t, q, e)
        v = new(len(t), d_in, t=F32)
        gpu_lib.mxfp4_dequantize(q, e, v)
        ops.append((q, e, v))
    (xq, x_e, xv), (wq, w_e, wv) = ops
    y, z = new(tokens, d_out, t=BF16), new(tokens, d_out, t=BF16)
    gpu_lib.melded_linear_fwd_mxfp4(xq, x_e, wq, w_e, y, act="relu", z=z)
    for at in (0, min(2 ** 31 // d_out, tokens - 60) - 20, tokens - 40):
        s = slice(at, at + 40)
        ref, S = xv[s].double() @ wv.double().T, xv[s].abs().double() @ wv.abs().double().T
        tol = S * 64 * 2.0 ** -24 + ref.abs() * 2.0 ** -8
        assert bool(((z[s] - ref).abs() <= tol).all())
        assert torch.equal(y[s], z[s].clamp(min=0))


def test_cross_entropy_of_far_tokens(gpu_lib):
    """2.3e9 codes of tokens, in nine strips; the last strip is short."""
    n, d, V = 140000, 16400, 70
    x = filled(n, d).to(torch.float8_e4m3fn)                # within 13 * 6 of 448
    wq = (torch.empty((V, d), device="cuda").normal_() * 64).to(torch.float8_e4m3fn)
    s_x, s_w = torch.tensor([1.0], device="cuda"), torch.tensor([64 * math.sqrt(d)], device="cuda")
    target = torch.arange(n, device="cuda") % V
    loss, lse = new(n, t=F32), new(n, t=F32)
    gpu_lib.linear_cross_entropy_fwd(x.view(U8), s_x, wq.view(U8), s_w, target, loss, lse)
    dloss, dx = torch.ones(n, device="cuda"), new(n, d, t=BF16)
    gpu_lib.linear_cross_entropy_bwd(x.view(U8), s_x, wq.view(U8), s_w, target, lse, dloss, dx)
    for at in (0, 2 ** 31 // d - 20, n - 40):
        s = slice(at, at + 40)
        k = 1 / float(s_w)
        z = x[s].double() @ wq.double().T * k
        S = x[s].double().abs() @ wq.double().abs().T * k
        ref = torch.logsumexp(z, 1)
        t = target[s, None]
        e = S.amax(1) * ((d / 4 + 8) * 2.0 ** -24) + 1e-5
        assert bool(((lse[s] - ref).abs() <= e).all())
        assert bool(((loss[s] - ref + z.gather(1, t)[:, 0]).abs() <= 2 * e).all())
        G = torch.exp(z - ref[:, None])
        G.scatter_(1, t, G.gather(1, t) - 1)
        want = G @ wq.double() * k
        # p off by expm1 of its logit's error (2^-13 of the largest of eight products, an
        # eighth of S or less each), G and dx by half a step each
        aw = wq.double().abs() * k
        rel = torch.expm1(S * 2.0 ** -13 + e[:, None]) + 2.0 ** -11
        tol = (G.abs() * rel) @ aw + (G.abs() @ aw) * (V * 2.0 ** -24) + want.abs() * 2.0 ** -8
        assert bool(((dx[s] - want).abs() <= tol + 2.0 ** -40 * aw.sum(0)).all())


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("tokens,d_out", [(8192, 8208), (8200, 16400)])
def test_float32_outputs_past_the_caches(gpu_lib, fp4, tokens, d_out):
    """269 MB of float32 and 1.1 GB of it, y and z, of the FP8 and the FP4 product with a
    bias; 64 products each, off by 64 half steps of their absolute sum at most, the bias's
    by one of the result."""
    d_in = 64
    x, w = filled(tokens, d_in, F32), filled(d_out, d_in, F32)
    bias = new(d_out, t=F32).normal_()
    y = new(tokens, d_out, t=F32)
    z = new(tokens, d_out, t=F32) if d_out > 10000 else None
    one = torch.ones(1, device="cuda")
    if fp4:
        ops, vals = [], []
        for t in (x, w):
            q, e = new(len(t), d_in // 2), new(*gpu_lib.mxfp4_scales_shape(len(t), d_in))
            gpu_lib.mxfp4_quantize(t, q, e)
            vals.append(new(len(t), d_in, t=F32))
            gpu_lib.mxfp4_dequantize(q, e, vals[-1])
            ops += [q, e]
        gpu_lib.melded_linear_fwd_mxfp4(*ops, y, bias=bias, act="relu", z=z)
    else:
        q = [t.to(torch.float8_e4m3fn) for t in (x, w)]
        vals = [t.float() for t in q]
        gpu_lib.melded_linear_fwd_act(q[0].view(U8), one, q[1].view(U8), one, y, bias=bias,
                                      act="relu", z=z)
    for at in (0, tokens // 2 - 20, tokens - 40):
        s = slice(at, at + 40)
        ref = vals[0][s].double() @ vals[1].double().T
        S = vals[0][s].abs().double() @ vals[1].abs().double().T
        # (of E4M3's products the matrix core cuts what lies 2^-13 below the largest of eight)
        tol = S * 64 * U + (S * 2.0 ** -13 if not fp4 else 0)
        ref = ref + bias.double()
        tol = tol + ref.abs() * U
        if z is not None:
            assert bool(((z[s] - ref).abs() <= tol).all())
        assert bool(((y[s] - ref.clamp(min=0)).abs() <= tol).all())
