"""The microscaled formats, the 8-bit checkpoints and the cross entropy refuse bad
arguments before anything is launched (these calls never reach the GPU, so they run on
a host without one)."""
import pytest
import torch

import fp8_quantized_lora_amd as fq

EINVAL, OK = 1, 0
P, Q, R, S, V, W = (1 << k for k in range(40, 46))   # fake addresses, never dereferenced
MIS = P + 1
U8, F32, BF16 = torch.uint8, torch.float32, torch.bfloat16


def refused(f, ok, changes):
    for idx, val in changes:
        a = list(ok)
        a[idx] = val
        assert f(*a) == EINVAL, (f.__name__, idx, val)


def test_mxfp4_formats():
    lib = fq.load()
    assert fq.mxfp4_scale_bytes(1, 32) == 128 and fq.mxfp4_scale_bytes(17, 288) == 2 * 32 * 8
    assert fq.mxfp4_scale_bytes(4, 33) == 0 and fq.mxfp4_scale_bytes(-1, 32) == 0
    #     x  t  rows K  q  e  stream
    ok = [P, 1, 4, 64, Q, R, None]
    refused(lib.mxfp4_quantize, ok, [(0, None), (0, MIS), (1, 2), (2, -1), (3, 48), (3, -32),
                                     (2, (1 << 30) + 1), (4, None), (4, Q + 8), (5, None),
                                     (5, R + 8), (4, P), (5, Q), (5, P)])
    #     q  e  rows K  x  t  stream
    ok = [Q, R, 4, 64, P, 0, None]
    refused(lib.mxfp4_dequantize, ok, [(0, None), (0, Q + 8), (1, None), (1, R + 8), (4, None),
                                       (4, P + 2), (5, 2), (3, 40), (4, Q), (4, R)])
    assert lib.mxfp4_quantize(None, 0, 0, 64, None, None, None) == OK
    assert lib.mxfp4_dequantize(None, None, 4, 0, None, 0, None) == OK


def test_mxfp4_product():
    lib = fq.load()
    f = lib.melded_linear_fwd_mxfp4
    assert fq.melded_linear_fwd_mxfp4_workspace_bytes(8, 64, 48) == 0
    assert fq.melded_linear_fwd_mxfp4_workspace_bytes(8, 48, 48) == 0
    nb = fq.melded_linear_fwd_mxfp4_workspace_bytes(129, 27648, 528)
    assert nb >= 2 * 129 * 528 * 4
    #     xq xe wq we b  act res T    di     do   t  y  z  ws n  stream
    ok = [P, Q, R, S, V, 2, None, 129, 27648, 528, 1, W, None, 1 << 46, nb, None]
    refused(f, ok, [(13, None), (13, (1 << 46) + 16), (14, nb - 1)])
    ok = [P, Q, R, S, V, 2, 1 << 47, 8, 64, 48, 1, W, 1 << 48, None, 0, None]
    refused(f, ok, [(0, None), (0, MIS), (1, None), (1, Q + 8), (2, None), (2, R + 8), (3, None),
                    (3, S + 8), (4, V + 2), (5, -1), (5, 5), (6, W + 2), (7, -1), (8, 48), (9, 40),
                    (10, 2), (11, None), (11, W + 1), (11, P), (11, S), (12, W), (12, Q),
                    (7, 1 << 31)])
    assert f(None, None, R, S, None, 0, None, 0, 64, 48, 1, None, None, None, 0, None) == OK
    assert f(P, Q, None, None, None, 0, None, 4, 64, 0, 1, None, None, None, 0, None) == OK


def test_checkpoints():
    lib = fq.load()
    #     x  t  T  d   q  e  stream
    ok = [P, 1, 4, 33, Q, R, None]
    refused(lib.checkpoint_save, ok, [(0, None), (0, MIS), (1, 2), (2, -1), (3, 0), (2, 1 << 31),
                                      (3, (1 << 24) + 1), (4, None), (5, None), (4, P), (5, P),
                                      (5, Q + 131), (4, R - 131)])
    ok = [Q, R, 4, 33, P, 0, None]
    refused(lib.checkpoint_restore, ok, [(0, None), (1, None), (4, None), (4, P + 2), (5, 2),
                                         (2, -1), (3, 0), (4, Q), (4, R)])
    assert lib.checkpoint_save(None, 0, 0, 33, None, None, None) == OK
    assert lib.checkpoint_restore(None, None, 0, 33, None, 0, None) == OK


def test_backwards_from_checkpoints():
    lib = fq.load()
    ws = fq.linear_act_bwd_workspace_bytes(1000, 48)
    #     dy t  zq ze act T   d   dz db ws n  stream
    ok = [P, 0, Q, R, 2, 1000, 48, S, V, W, ws, None]
    refused(lib.linear_act_bwd_ckpt, ok, [(0, None), (0, P + 2), (1, 2), (2, None), (3, None),
                                          (4, -1), (4, 5), (5, -1), (6, 0), (6, (1 << 24) + 1),
                                          (7, S + 2), (7, Q), (7, P + 4), (8, V + 2), (8, R),
                                          (9, None), (9, W + 16), (10, ws - 1)])
    assert lib.linear_act_bwd_ckpt(P, 0, Q, R, 2, 4, 48, None, None, None, 0, None) == EINVAL
    ws = fq.layer_norm_bwd_workspace_bytes(2000, 64)
    #     dy t  xq xe w     mu       rs       T     d   dx dw       db       ws n  stream
    ok = [P, 1, Q, R, None, 1 << 46, 1 << 47, 2000, 64, S, 1 << 48, 1 << 49, W, ws, None]
    refused(lib.layer_norm_bwd_ckpt, ok, [(0, None), (0, MIS), (1, 2), (2, None), (3, None),
                                          (4, V + 2), (5, None), (6, None), (7, -1), (8, 0),
                                          (9, S + 1), (9, Q), (9, R), (10, P), (11, 1 << 48),
                                          (12, None), (12, W + 16), (13, ws - 1)])


def test_cross_entropy():
    lib = fq.load()
    n = fq.linear_cross_entropy_fwd_workspace_bytes(20, 64, 1000)
    assert n >= 20 * 4 and fq.linear_cross_entropy_fwd_workspace_bytes(20, 72, 1000) == 0
    assert fq.linear_cross_entropy_fwd_workspace_bytes(20, 64, 0) == 0
    T, A, B = 1 << 46, 1 << 47, 1 << 48
    #     xq sx wq sw t  T   d   V     loss lse ws n stream
    ok = [P, Q, R, S, T, 20, 64, 1000, A, B, V, n, None]
    common = [(0, None), (0, P + 8), (1, None), (1, Q + 2), (2, None), (2, R + 8), (3, None),
              (3, S + 2), (4, None), (4, T + 4)]
    refused(lib.linear_cross_entropy_fwd, ok,
            common + [(5, -1), (6, 0), (6, 72), (6, (1 << 22) + 16), (7, 0), (7, (1 << 22) + 1),
                      (8, None), (8, A + 2), (9, B + 2), (9, A), (8, T), (8, P), (9, R), (10, None),
                      (10, V + 16), (11, n - 1)])
    for dt, t in ((torch.float32, 0), (torch.bfloat16, 1)):
        m = fq.linear_cross_entropy_bwd_workspace_bytes(20, 64, 1000, dt)
        assert m > 0
        #     xq sx wq sw t  lse dl T  d   V     dx t  ws n stream
        ok = [P, Q, R, S, T, A, B, 20, 64, 1000, W, t, V, m, None]
        refused(lib.linear_cross_entropy_bwd, ok,
                common + [(5, None), (5, A + 2), (6, None), (7, -1), (8, 8), (9, 0), (10, None),
                          (10, W + 1), (10, P), (10, R), (10, T), (10, A), (10, B), (11, 2),
                          (12, None), (12, V + 16), (13, m - 1)])
    assert lib.linear_cross_entropy_fwd(None, Q, R, S, None, 0, 64, 9, None, None, None, 0,
                                        None) == OK
    assert lib.linear_cross_entropy_bwd(None, Q, R, S, None, None, None, 0, 64, 9, None, 0, None,
                                        0, None) == OK


def test_workspaces_do_not_grow_beyond_a_strip():
    a = fq.linear_cross_entropy_bwd_workspace_bytes(16384, 4096, 131072, torch.bfloat16)
    assert fq.linear_cross_entropy_bwd_workspace_bytes(1 << 20, 4096, 131072, torch.bfloat16) == a
    # far from the logits themselves: 16384 x 131072 float32 are 8 GB
    assert a < 1 << 30
    # every size that is taken has a workspace
    for T in (1, 16, 17, 300, 16384, 16385, 16400, 40000):
        for d in (16, 4096, 1 << 22):
            for n in (1, 1000, 131071, 1 << 22):
                assert fq.linear_cross_entropy_fwd_workspace_bytes(T, d, n) > 0
                assert fq.linear_cross_entropy_bwd_workspace_bytes(T, d, n) > 0


# ---------------------------------------------------------------------------
# the binding's checks, each by its message
class Made:
    def __init__(self, dev):
        self.dev = dev

    def __call__(self, *shape, dtype=F32):
        return torch.zeros(shape, dtype=dtype, device=self.dev)


def quantize(t, **k):
    fq.mxfp4_quantize(**{**dict(x=t(4, 64), q=t(4, 32, dtype=U8), e=t(1, 16, 8, dtype=U8)), **k})


def dequantize(t, **k):
    fq.mxfp4_dequantize(**{**dict(x=t(4, 64), q=t(4, 32, dtype=U8), e=t(1, 16, 8, dtype=U8)), **k})


def product(t, **k):
    a = dict(xq=t(4, 32, dtype=U8), x_e=t(1, 16, 8, dtype=U8), wq=t(48, 32, dtype=U8),
             w_e=t(1, 48, 8, dtype=U8), y=t(4, 48), bias=t(48), act="gelu", residual=t(4, 48),
             z=t(4, 48))
    fq.melded_linear_fwd_mxfp4(**{**a, **k})


def save(t, **k):
    fq.checkpoint_save(**{**dict(x=t(4, 33), q=t(4, 33, dtype=U8), e=t(4, 2, dtype=U8)), **k})


def restore(t, **k):
    fq.checkpoint_restore(**{**dict(x=t(4, 33), q=t(4, 33, dtype=U8), e=t(4, 2, dtype=U8)), **k})


def act_bwd(t, **k):
    a = dict(dy=t(4, 33), z_q=t(4, 33, dtype=U8), z_e=t(4, 2, dtype=U8), dz=t(4, 33), dbias=t(33),
             act="gelu")
    fq.linear_act_bwd_ckpt(**{**a, **k})


def norm_bwd(t, **k):
    a = dict(dy=t(4, 33), x_q=t(4, 33, dtype=U8), x_e=t(4, 2, dtype=U8), weight=t(33), mean=t(4),
             rstd=t(4), dx=t(4, 33), dweight=t(33), dbias=t(33))
    fq.layer_norm_bwd_ckpt(**{**a, **k})


def loss_fwd(t, **k):
    a = dict(xq=t(4, 32, dtype=U8), s_x=t(1), wq=t(9, 32, dtype=U8), s_w=t(1),
             target=t(4, dtype=torch.int64), loss=t(4), lse=t(4))
    fq.linear_cross_entropy_fwd(**{**a, **k})


def loss_bwd(t, **k):
    a = dict(xq=t(4, 32, dtype=U8), s_x=t(1), wq=t(9, 32, dtype=U8), s_w=t(1),
             target=t(4, dtype=torch.int64), lse=t(4), dloss=t(4), dx=t(4, 32))
    fq.linear_cross_entropy_bwd(**{**a, **k})


CALLS = (quantize, dequantize, product, save, restore, act_bwd, norm_bwd, loss_fwd, loss_bwd)
I32, F16, F64 = torch.int32, torch.float16, torch.float64
CASES = [
    (quantize, lambda t: dict(x=t(4, 48)), "^x: rows must be whole blocks of 32"),
    (quantize, lambda t: dict(x=t(4, 64, dtype=F16)), "^x: expected float32 or bfloat16"),
    (quantize, lambda t: dict(x=t(256)), "^x: expected two dimensions"),
    (quantize, lambda t: dict(x=t(64, 4).T), "contiguous"),
    (quantize, lambda t: dict(q=t(4, 64, dtype=U8)), "^q: expected shape"),
    (quantize, lambda t: dict(q=t(4, 32, dtype=torch.int8)), "^q: expected dtype"),
    (quantize, lambda t: dict(e=t(4, 2, dtype=U8)), "^e: expected shape"),
    (quantize, lambda t: dict(e=t(1, 16, 8)), "^e: expected dtype"),
    (dequantize, lambda t: dict(x=t(4, 96)), "^q: expected shape"),
    (dequantize, lambda t: dict(x=t(4, 64, dtype=F64)), "^x: expected float32 or bfloat16"),
    (dequantize, lambda t: dict(e=t(1, 32, 8, dtype=U8)), "^e: expected shape"),
    (product, lambda t: dict(xq=t(4, 24, dtype=U8)), "^xq: rows must be whole blocks"),
    (product, lambda t: dict(x_e=t(1, 48, 8, dtype=U8)), "^x_e: expected shape"),
    (product, lambda t: dict(w_e=t(1, 16, 8, dtype=U8)), "^w_e: expected shape"),
    (product, lambda t: dict(wq=t(48, 48, dtype=U8)), "^wq: expected shape"),
    (product, lambda t: dict(y=t(4, 47)), "^y: expected shape"),
    (product, lambda t: dict(y=t(4, 48, dtype=F16)), "^y: expected float32 or bfloat16"),
    (product, lambda t: dict(z=t(4, 48, dtype=BF16)), "^z: expected dtype"),
    (product, lambda t: dict(residual=t(48, 4).T), "contiguous"),
    (product, lambda t: dict(bias=t(4)), "^bias: expected shape"),
    (product, lambda t: dict(act="tanh"), "^act must be one of"),
    (save, lambda t: dict(q=t(4, 32, dtype=U8)), "^q: expected shape"),
    (save, lambda t: dict(e=t(4, 1, dtype=U8)), "^e: expected shape"),
    (save, lambda t: dict(x=t(4, 33, dtype=F16)), "^x: expected float32 or bfloat16"),
    (restore, lambda t: dict(q=t(33, 4, dtype=U8).T), "contiguous"),
    (restore, lambda t: dict(e=t(2, 4, dtype=U8)), "^e: expected shape"),
    (act_bwd, lambda t: dict(z_q=t(4, 33)), "^z_q: expected dtype"),
    (act_bwd, lambda t: dict(z_e=t(4, 3, dtype=U8)), "^z_e: expected shape"),
    (act_bwd, lambda t: dict(dz=t(4, 33, dtype=BF16)), "^dz: expected dtype"),
    (act_bwd, lambda t: dict(dbias=t(4)), "^dbias: expected shape"),
    (act_bwd, lambda t: dict(act=3), "^act must be one of"),
    (norm_bwd, lambda t: dict(x_q=t(3, 33, dtype=U8)), "^x_q: expected shape"),
    (norm_bwd, lambda t: dict(x_e=t(4, 2)), "^x_e: expected dtype"),
    (norm_bwd, lambda t: dict(mean=t(3)), "^mean: expected shape"),
    (norm_bwd, lambda t: dict(dx=t(4, 33, dtype=BF16)), "^dx: expected dtype"),
    (norm_bwd, lambda t: dict(weight=t(33, dtype=BF16)), "^weight: expected dtype"),
    (loss_fwd, lambda t: dict(target=t(4, dtype=I32)), "^target: expected dtype"),
    (loss_fwd, lambda t: dict(target=t(5, dtype=torch.int64)), "^target: expected shape"),
    (loss_fwd, lambda t: dict(wq=t(9, 16, dtype=U8)), "^wq: expected shape"),
    (loss_fwd, lambda t: dict(s_x=t(4)), "^s_x: expected shape"),
    (loss_fwd, lambda t: dict(loss=t(4, dtype=BF16)), "^loss: expected dtype"),
    (loss_fwd, lambda t: dict(lse=t(4, 1)), "^lse: expected shape"),
    (loss_bwd, lambda t: dict(dx=t(4, 32, dtype=F16)), "^dx: expected float32 or bfloat16"),
    (loss_bwd, lambda t: dict(dx=t(32, 4).T), "contiguous"),
    (loss_bwd, lambda t: dict(dloss=t(1)), "^dloss: expected shape"),
    (loss_bwd, lambda t: dict(lse=t(4, dtype=F64)), "^lse: expected dtype"),
]


def host_ptr(t):
    if not t.is_contiguous():
        raise fq.FalqError("tensor arguments must be contiguous")


@pytest.mark.parametrize("call, change, message", CASES)
def test_on_the_host(monkeypatch, call, change, message):
    monkeypatch.setattr(fq, "_device", lambda t, name: t.get_device())
    monkeypatch.setattr(fq, "_stream_of", lambda dev, stream: 0)
    monkeypatch.setattr(fq, "_run", lambda *a: pytest.fail("the library was called"))
    monkeypatch.setattr(fq, "_ptr", host_ptr)
    t = Made("cpu")
    with pytest.raises(fq.FalqError, match=message):
        call(t, **change(t))


def test_the_calls_as_they_are_would_run(monkeypatch):
    """Unchanged, each call passes every check and reaches the library."""
    ran = []
    monkeypatch.setattr(fq, "_device", lambda t, name: t.get_device())
    monkeypatch.setattr(fq, "_stream_of", lambda dev, stream: 0)
    monkeypatch.setattr(fq, "_run", lambda fn, what, *a: ran.append(what))
    monkeypatch.setattr(fq, "_scratch", lambda *a: None)
    for call in CALLS:
        call(Made("cpu"))
    assert ran == ["mxfp4_quantize", "mxfp4_dequantize", "melded_linear_fwd_mxfp4",
                   "checkpoint_save", "checkpoint_restore", "linear_act_bwd_ckpt",
                   "layer_norm_bwd_ckpt", "linear_cross_entropy_fwd", "linear_cross_entropy_bwd"]


def test_tensors_on_the_host_are_refused():
    for call in CALLS:
        with pytest.raises(fq.FalqError, match="GPU|cuda"):
            call(Made("cpu"))


@pytest.mark.gpu
@pytest.mark.parametrize("call, change, message", CASES)
def test_on_the_gpu(gpu_lib, monkeypatch, call, change, message):
    monkeypatch.setattr(fq, "_run", lambda *a: pytest.fail("the library was called"))
    t = Made("cuda")
    with pytest.raises(fq.FalqError, match=message):
        call(t, **change(t))


def test_layers():
    cpu = dict(device="cpu")
    bad = pytest.raises(ValueError)
    with bad:
        fq.MeldedLinear(32, 32, 4, 8, act="gelu", keep_z="half", **cpu)
    with bad:
        fq.MeldedLinear(32, 32, 4, 8, bias=True, keep_z="fp8", **cpu)
    with bad:
        fq.MeldedLinear(32, 32, 4, 8, act="gelu", z_scratch=torch.zeros(256), **cpu)
    for z in (torch.zeros(255), torch.zeros(256, dtype=BF16), torch.zeros(512)[::2]):
        with bad:
            fq.MeldedLinear(32, 32, 4, 8, act="gelu", keep_z="fp8", z_scratch=z, **cpu)
    z = torch.zeros(300)
    m = fq.MeldedLinear(32, 32, 4, 8, act="gelu", keep_z="fp8", z_scratch=z, **cpu)
    assert m.z.data_ptr() == z.data_ptr() and m.z_q.shape == (8, 32) and m.z_e.shape == (8, 1)
    with bad:
        fq.LinearCrossEntropy(100, 32, 8, dx_dtype=F16, **cpu)
    assert fq.LinearCrossEntropy(100, 32, 8, dx_dtype=BF16, **cpu).dx.dtype == BF16
