"""FP4 operands (mxfp4_quantize, mxfp4_dequantize) and 8-bit checkpoints
(checkpoint_save, checkpoint_restore) bit for bit against their definitions: scaling by
a power of two is exact, so every element is rounded once and there is no tolerance."""
import numpy as np
import pytest
import torch

from tests import mx_ref as ref
from tests.gpu_util import announce, dev, host

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U8 = torch.uint8


def values(rows, n, kind, seed=0):
    rng = np.random.default_rng(seed + rows * 7 + n)
    x = rng.standard_normal((rows, n)).astype(np.float32)
    if kind == "wide":                            # every binade
        x *= np.exp2(rng.integers(-126, 125, (rows, n))).astype(np.float32)
    elif kind == "tiny":                          # subnormal and zero blocks
        x *= np.float32(2.0 ** -140)
        x[:, ::3] = 0
        x[rows // 2] = 0
    elif kind == "ties":                          # halfway between codes of either format
        m = rng.choice(np.concatenate([(ref.E2M1[1:] + ref.E2M1[:-1]) / 2, ref.E2M1,
                                       (ref.E4M3[1:] + ref.E4M3[:-1]) / 2, ref.E4M3, [7, 448, 480]]),
                       (rows, n))
        x = (m * rng.choice([-1, 1], (rows, n))).astype(np.float32)
        x[:, ::32] = np.where(rng.random((rows, len(range(0, n, 32)))) < .5, 4, 448)
    elif kind == "special":
        x *= 30
        x.flat[rng.integers(0, x.size, x.size // 5 + 1)] = np.nan
        x.flat[rng.integers(0, x.size, x.size // 5 + 1)] = np.inf
        x.flat[rng.integers(0, x.size, x.size // 5 + 1)] = -np.inf
        x.flat[rng.integers(0, x.size, x.size // 9 + 1)] = -0.0
        x[-1] = np.nan                            # nothing finite in these blocks
    return x


def typed(x, dtype):
    t = dev(x).to(dtype)
    return t, host(t.float()).astype(np.float64)


KINDS = ("plain", "wide", "tiny", "ties", "special")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows, K", [(1, 32), (3, 64), (16, 256), (17, 288), (33, 4064), (130, 544)])
def test_mxfp4(gpu_lib, rows, K, kind, dtype):
    announce(f"mxfp4_quantize {rows} x {K} {kind} {dtype}")
    x, v = typed(values(rows, K, kind), dtype)
    q = torch.full((rows, K // 2), 0x55, dtype=U8, device="cuda")
    e = torch.full(gpu_lib.mxfp4_scales_shape(rows, K), 0x55, dtype=U8, device="cuda")
    assert e.numel() == gpu_lib.mxfp4_scale_bytes(rows, K)
    gpu_lib.mxfp4_quantize(x, q, e)
    c, ex = ref.encode(v, "fp4")
    assert np.array_equal(host(e), ref.pack_exponents(ex))
    assert np.array_equal(host(q), ref.pack4(c))
    for out in (F32, BF16):
        y = torch.full((rows, K), 9.0, dtype=out, device="cuda")
        gpu_lib.mxfp4_dequantize(q, e, y)
        want = torch.from_numpy(ref.decode(c, ex, "fp4")).to(out)
        assert torch.equal(y.cpu(), want)
        assert torch.equal(torch.signbit(y.cpu()), torch.signbit(want))


def test_every_code_and_exponent(gpu_lib):
    """All sixteen codes under all 256 exponent bytes."""
    rows, K = 256, 32
    q = dev(np.tile(ref.pack4(np.tile(np.arange(16, dtype=np.uint8), 2)[None]), (rows, 1)))
    e = np.full((1, rows, 8), 127, np.uint8)
    e[0, :, 0] = np.arange(rows)
    y = torch.empty((rows, K), device="cuda")
    gpu_lib.mxfp4_dequantize(q, dev(e), y)
    want = ref.decode(ref.unpack4(host(q)), np.arange(-127, 129)[:, None], "fp4")
    with np.errstate(over="ignore"):
        assert np.array_equal(host(y), want.astype(np.float32), equal_nan=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T, d", [(1, 1), (3, 7), (2, 31), (5, 32), (4, 33), (16, 40), (7, 1000),
                                  (33, 1027), (130, 400), (1, 20000)])
def test_checkpoint(gpu_lib, T, d, kind, dtype):
    announce(f"checkpoint_save {T} x {d} {kind} {dtype}")
    x, v = typed(values(T, d, kind), dtype)
    q = torch.full((T, d), 0x55, dtype=U8, device="cuda")
    e = torch.full(gpu_lib.checkpoint_scales_shape(T, d), 0x55, dtype=U8, device="cuda")
    gpu_lib.checkpoint_save(x, q, e)
    c, ex = ref.encode(v, "fp8")
    assert np.array_equal(host(e), (ex + 127).astype(np.uint8))
    assert np.array_equal(host(q), c)
    for out in (F32, BF16):
        y = torch.full((T, d), 9.0, dtype=out, device="cuda")
        gpu_lib.checkpoint_restore(q, e, y)
        want = torch.from_numpy(ref.decode(c, ex, "fp8")).to(out)
        assert torch.equal(torch.isnan(y.cpu()), torch.isnan(want))
        assert torch.equal(y.cpu().nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))


def test_rows_anywhere_in_a_buffer(gpu_lib):
    """Elements, codes and exponents need only their own alignment, and what lies
    before and behind the outputs is left alone."""
    T, d = 9, 45
    buf = torch.zeros(T * d + 8, dtype=BF16, device="cuda")
    x = buf[3: 3 + T * d].view(T, d)
    x.copy_(dev(values(T, d, "plain")))
    nb = (d + 31) // 32
    qb = torch.full((T * d + 8,), 0xAA, dtype=U8, device="cuda")
    eb = torch.full((T * nb + 8,), 0xAA, dtype=U8, device="cuda")
    q, e = qb[5: 5 + T * d].view(T, d), eb[1: 1 + T * nb].view(T, nb)
    gpu_lib.checkpoint_save(x, q, e)
    c, ex = ref.encode(host(x.float()).astype(np.float64), "fp8")
    assert np.array_equal(host(q), c) and np.array_equal(host(e), (ex + 127).astype(np.uint8))
    for b, o, n in ((qb, 5, T * d), (eb, 1, T * nb)):
        assert bool((b[:o] == 0xAA).all()) and bool((b[o + n:] == 0xAA).all())
    y = torch.zeros(T * d + 8, device="cuda")
    gpu_lib.checkpoint_restore(q, e, y[1: 1 + T * d].view(T, d))
    assert np.array_equal(host(y)[1: 1 + T * d].reshape(T, d), ref.decode(c, ex, "fp8"))
    assert float(y[0]) == 0 and not bool(y[1 + T * d:].any())


def test_no_rows(gpu_lib):
    x = torch.empty((0, 64), device="cuda")
    gpu_lib.mxfp4_quantize(x, torch.empty((0, 32), dtype=U8, device="cuda"),
                           torch.empty(gpu_lib.mxfp4_scales_shape(0, 64), dtype=U8, device="cuda"))
    gpu_lib.checkpoint_save(x, torch.empty((0, 64), dtype=U8, device="cuda"),
                            torch.empty((0, 2), dtype=U8, device="cuda"))
    gpu_lib.checkpoint_restore(torch.empty((0, 64), dtype=U8, device="cuda"),
                               torch.empty((0, 2), dtype=U8, device="cuda"), x)
