"""Tensors of more than 2^31 elements: rows past a 32-bit offset are read and
written where they belong.  Rows of these operators do not depend on each other
(the sums over rows aside), so the last rows are checked against the same rows
in a call of their own, within half a step of bfloat16 twice (2^-7: two
roundings of values that differ by float32 roundings at most)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
T, D, TAIL = 270_000, 8192, 500                      # 2.2e9 elements


def close(a, b):
    a, b = a.float(), b.float()
    return bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-3 * b.abs().max()).all())


@pytest.fixture(scope="module")
def big():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.empty((T, D), dtype=BF16, device="cuda")
    x.normal_(generator=g)
    assert x.numel() > 2 ** 31
    yield x
    del x
    torch.cuda.empty_cache()


def test_layer_norm(gpu_lib, big):
    w, b = torch.randn(D, device="cuda"), torch.randn(D, device="cuda")
    y = torch.empty_like(big)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    gpu_lib.layer_norm_fwd(big, w, b, y, mean, rstd)
    x = big[-TAIL:].contiguous()
    y2, m2, r2 = torch.empty_like(x), *(torch.empty(TAIL, device="cuda") for _ in range(2))
    gpu_lib.layer_norm_fwd(x, w, b, y2, m2, r2)
    assert close(y[-TAIL:], y2) and close(mean[-TAIL:], m2) and close(rstd[-TAIL:], r2)
    # backward, dy = x, dx in y's memory
    dw, db = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    gpu_lib.layer_norm_bwd(big, big, w, mean, rstd, y, dw, db)
    gpu_lib.layer_norm_bwd(x, x, w, m2, r2, y2)
    assert close(y[-TAIL:], y2)
    ref = torch.zeros(D, dtype=torch.float64, device="cuda")
    for part in big.split(30_000):
        ref += part.double().sum(0)
    # 2.7e5 standard normals: a chain of at most T roundings of sums below 5 sqrt(T)
    assert float((db.double() - ref).abs().max()) <= T * 2.0 ** -24 * 5 * math.sqrt(T)


def test_activation_backward(gpu_lib, big):
    dz, db = torch.empty_like(big), torch.empty(D, device="cuda")
    gpu_lib.linear_act_bwd(big, big, dz, dbias=db, act="silu")
    x = big[-TAIL:].contiguous()
    z2 = torch.empty_like(x)
    gpu_lib.linear_act_bwd(x, x, z2, act="silu")
    assert close(dz[-TAIL:], z2)


def test_product(gpu_lib):
    xq = torch.randint(0, 120, (T, 64), dtype=torch.uint8, device="cuda")
    wq = torch.randint(0, 120, (D, 64), dtype=torch.uint8, device="cuda")
    one, bias = torch.ones(1, device="cuda"), torch.randn(D, device="cuda")
    y = torch.empty((T, D), dtype=BF16, device="cuda")
    gpu_lib.melded_linear_fwd_act(xq, one, wq, one, y, bias=bias, act="relu")
    x = xq[-TAIL:].contiguous()
    y2 = torch.empty((TAIL, D), dtype=BF16, device="cuda")
    gpu_lib.melded_linear_fwd_act(x, one, wq, one, y2, bias=bias, act="relu")
    assert close(y[-TAIL:], y2)


def test_clip(gpu_lib, big):
    flat = big.view(-1)
    n = flat.numel()
    views = [flat[1:n - 7], flat[n - 5:]]
    out = torch.empty_like(flat)
    norm = torch.empty(1, device="cuda")
    gpu_lib.grad_clip(views, 1.0, norm, out=[out[1:n - 7], out[n - 5:]])
    ref = math.sqrt(sum(float(p.double().square().sum()) for p in flat.split(2 ** 28)))
    assert abs(float(norm) / ref - 1) <= 1e-6        # three elements are left out
    want = flat[-1000:].float() / float(norm)
    got = out[-1000:].float()
    keep = torch.ones(1000, dtype=torch.bool, device="cuda")
    keep[-7:-5] = False                              # between the views
    assert bool(((got - want).abs() <= 2.0 ** -7 * want.abs())[keep].all())


@pytest.mark.parametrize("T, d_in, d_out", [(4096, 1 << 23, 5120), (40, (1 << 23) + 144, 64),
                                            (3, (1 << 23) + 144, 64)])
def test_product_over_long_rows(gpu_lib, T, d_in, d_out):
    """Rows so long that a tile's last ones begin 2^31 bytes behind its first, and
    rows past what the larger tiles' offsets reach.  Codes of +-1: every sum is an
    integer below 2^24, exact in float32."""
    g = torch.Generator(device="cuda")
    g.manual_seed(9)

    def signs(rows):
        t = torch.empty((rows, d_in), dtype=torch.uint8, device="cuda")
        t.random_(0, 2, generator=g)
        return t.mul_(128).bitwise_or_(0x38)

    xq, wq = signs(T), signs(d_out)
    one = torch.ones(1, device="cuda")
    y = torch.empty((T, d_out), device="cuda")
    gpu_lib.melded_linear_fwd_act(xq, one, wq, one, y)
    rows = sorted({0, 1, T // 2, T - 1})
    ref = torch.zeros((len(rows), d_out), dtype=torch.float64, device="cuda")
    for a in range(0, d_in, 1 << 16):
        x = xq[rows, a:a + (1 << 16)].view(torch.float8_e4m3fn).float()
        w = wq[:, a:a + (1 << 16)].contiguous().view(torch.float8_e4m3fn).float()
        ref += (x @ w.T).double()
    assert torch.equal(y[rows].double(), ref)
    del xq, wq
    torch.cuda.empty_cache()
