"""The binding's checks of shapes, types, contiguity and devices around the linear,
each by its message, so that each is the check that refuses: the kernels take raw
pointers, and nothing behind the binding knows a tensor's size.

On the CPU the device check is taken out of the way (the tensors stand for GPU
tensors; no call may reach the library); marked gpu, the same calls with GPU
tensors."""
import pytest
import torch

import fp8_quantized_lora_amd as fq

F32, BF16, U8, F16 = torch.float32, torch.bfloat16, torch.uint8, torch.float16


class Made:
    """Tensors by size, on one device."""

    def __init__(self, dev):
        self.dev = dev

    def __call__(self, *shape, dtype=F32):
        return torch.zeros(shape, dtype=dtype, device=self.dev)

    def strided(self, rows, cols, dtype=F32):
        return torch.zeros((rows, 2 * cols), dtype=dtype, device=self.dev)[:, :cols]


T, D, N = 4, 64, 48


def norm_fwd(t, **k):
    a = dict(x=t(T, D), weight=t(D), bias=t(D), y=t(T, D), mean=t(T), rstd=t(T))
    fq.layer_norm_fwd(**{**a, **k})


def norm_bwd(t, **k):
    a = dict(dy=t(T, D), x=t(T, D), weight=t(D), mean=t(T), rstd=t(T), dx=t(T, D), dweight=t(D),
             dbias=t(D))
    fq.layer_norm_bwd(**{**a, **k})


def product(t, **k):
    a = dict(xq=t(T, D, dtype=U8), s_x=t(1), wq=t(N, D, dtype=U8), s_w=t(1), y=t(T, N),
             bias=t(N), act="gelu", residual=t(T, N), z=t(T, N))
    fq.melded_linear_fwd_act(**{**a, **k})


def act_bwd(t, **k):
    a = dict(dy=t(T, N), z=t(T, N), dz=t(T, N), dbias=t(N), act="gelu")
    fq.linear_act_bwd(**{**a, **k})


def norm(t, **k):
    fq.grad_norm(**{**dict(grads=[t(5, 3), t(7)], norm=t(1)), **k})


def clip(t, **k):
    a = dict(grads=[t(5, 3), t(7)], max_norm=1.0, norm=t(1), out=[t(5, 3), t(7)])
    fq.grad_clip(**{**a, **k})


def shape(name, got):
    return rf"^{name}: expected shape .*, got {got}".replace("(", r"\(").replace(")", r"\)")


def dtype(name, got):
    return rf"^{name}: expected dtype .*, got torch.{got}"


LIST = "every tensor must be contiguous"
CASES = [
    (norm_fwd, lambda t: dict(x=t(T, D, dtype=F16)), "^x: expected float32 or bfloat16"),
    (norm_fwd, lambda t: dict(y=t(T, D, dtype=F16)), "^y: expected float32 or bfloat16"),
    (norm_fwd, lambda t: dict(x=t(T * D)), "^x: expected two dimensions"),
    (norm_fwd, lambda t: dict(x=t.strided(T, D)), "contiguous"),
    (norm_fwd, lambda t: dict(y=t.strided(T, D)), "contiguous"),
    (norm_fwd, lambda t: dict(y=t(T + 1, D)), shape("y", "(5, 64)")),
    (norm_fwd, lambda t: dict(y=t(T, D - 1)), shape("y", "(4, 63)")),
    (norm_fwd, lambda t: dict(weight=t(D - 1)), shape("weight", "(63,)")),
    (norm_fwd, lambda t: dict(weight=t(D, dtype=BF16)), dtype("weight", "bfloat16")),
    (norm_fwd, lambda t: dict(bias=t(2 * D)), shape("bias", "(128,)")),
    (norm_fwd, lambda t: dict(bias=t(2 * D)[::2]), "contiguous"),
    (norm_fwd, lambda t: dict(mean=t(T + 1)), shape("mean", "(5,)")),
    (norm_fwd, lambda t: dict(rstd=t(T - 1)), shape("rstd", "(3,)")),
    (norm_fwd, lambda t: dict(rstd=t(T, dtype=torch.float64)), dtype("rstd", "float64")),
    (norm_bwd, lambda t: dict(dy=t(T - 1, D)), shape("dy", "(3, 64)")),
    (norm_bwd, lambda t: dict(dy=t(T, D, dtype=F16)), "^dy: expected float32 or bfloat16"),
    (norm_bwd, lambda t: dict(x=t.strided(T, D)), "contiguous"),
    (norm_bwd, lambda t: dict(dx=t(T, D, dtype=BF16)), dtype("dx", "bfloat16")),
    (norm_bwd, lambda t: dict(dx=t(T, D + 4)), shape("dx", "(4, 68)")),
    (norm_bwd, lambda t: dict(weight=t(1)), shape("weight", "(1,)")),
    (norm_bwd, lambda t: dict(mean=t(1)), shape("mean", "(1,)")),
    (norm_bwd, lambda t: dict(rstd=t(2)), shape("rstd", "(2,)")),
    (norm_bwd, lambda t: dict(dweight=t(D - 16)), shape("dweight", "(48,)")),
    (norm_bwd, lambda t: dict(dbias=t(D, dtype=BF16)), dtype("dbias", "bfloat16")),
    (product, lambda t: dict(xq=t(T, D)), dtype("xq", "float32")),
    (product, lambda t: dict(xq=t(T, D + 16, dtype=U8)), shape("wq", "(48, 64)")),
    (product, lambda t: dict(xq=t.strided(T, D, dtype=U8)), "contiguous"),
    (product, lambda t: dict(wq=t(D, N, dtype=U8).T), "contiguous"),
    (product, lambda t: dict(wq=t(N, D, dtype=torch.int8)), dtype("wq", "int8")),
    (product, lambda t: dict(s_x=t(2)), shape("s_x", "(2,)")),
    (product, lambda t: dict(s_w=t(1, dtype=torch.float64)), dtype("s_w", "float64")),
    (product, lambda t: dict(y=t(T, N - 16)), shape("y", "(4, 32)")),
    (product, lambda t: dict(y=t(T, N, dtype=F16)), "^y: expected float32 or bfloat16"),
    (product, lambda t: dict(bias=t(N - 1)), shape("bias", "(47,)")),
    (product, lambda t: dict(residual=t(T, N, dtype=BF16)), dtype("residual", "bfloat16")),
    (product, lambda t: dict(residual=t(T - 1, N)), shape("residual", "(3, 48)")),
    (product, lambda t: dict(z=t(T, N, dtype=BF16)), dtype("z", "bfloat16")),
    (product, lambda t: dict(z=t(N, T)), shape("z", "(48, 4)")),
    (product, lambda t: dict(act="tanh"), "^act must be one of"),
    (product, lambda t: dict(act=["gelu"]), "^act must be one of"),
    (act_bwd, lambda t: dict(z=None), "^linear_act_bwd: z is needed"),
    (act_bwd, lambda t: dict(z=t(T - 2, N)), shape("z", "(2, 48)")),
    (act_bwd, lambda t: dict(z=t(T, N, dtype=F16)), "^z: expected float32 or bfloat16"),
    (act_bwd, lambda t: dict(dy=t(T, N, dtype=F16)), "^dy: expected float32 or bfloat16"),
    (act_bwd, lambda t: dict(dy=t(T * N)), "^dy: expected two dimensions"),
    (act_bwd, lambda t: dict(dz=t(T, N, dtype=BF16)), dtype("dz", "bfloat16")),
    (act_bwd, lambda t: dict(dz=t.strided(T, N)), "contiguous"),
    (act_bwd, lambda t: dict(dbias=t(N + 1)), shape("dbias", "(49,)")),
    (norm, lambda t: dict(norm=t(2)), shape("norm", "(2,)")),
    (norm, lambda t: dict(norm=t(1, dtype=torch.float64)), dtype("norm", "float64")),
    (norm, lambda t: dict(grads=[t(4), t(4, dtype=F16)]), "expected float32 or bfloat16"),
    (norm, lambda t: dict(grads=[t(4), t(8)[::2]]), LIST),
    (clip, lambda t: dict(norm=t(2)), shape("norm", "(2,)")),
    (clip, lambda t: dict(grads=[t(5, 3), t(7, dtype=torch.float64)]),
     "expected float32 or bfloat16"),
    (clip, lambda t: dict(grads=[t(3, 5).T, t(7)]), LIST),
    (clip, lambda t: dict(out=[t(5, 3)]), "1 outputs for 2 tensors"),
    (clip, lambda t: dict(out=[t(5, 3), t(6)]), "out must have the tensors' types and sizes"),
    (clip, lambda t: dict(out=[t(5, 3), t(7, dtype=BF16)]),
     "out must have the tensors' types and sizes"),
    (clip, lambda t: dict(out=[t(5, 3), t(14)[::2]]), LIST),
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
    for call in (norm_fwd, norm_bwd, product, act_bwd, norm, clip):
        call(Made("cpu"))
    assert ran == ["layer_norm_fwd", "layer_norm_bwd", "melded_linear_fwd_act", "linear_act_bwd",
                   "grad_norm", "grad_clip"]


@pytest.mark.gpu
@pytest.mark.parametrize("call, change, message", CASES)
def test_on_the_gpu(gpu_lib, monkeypatch, call, change, message):
    monkeypatch.setattr(fq, "_run", lambda *a: pytest.fail("the library was called"))
    t = Made("cuda")
    with pytest.raises(fq.FalqError, match=message):
        call(t, **change(t))


@pytest.mark.gpu
def test_a_tensor_on_the_host(gpu_lib, monkeypatch):
    """Each tensor of each call in turn."""
    monkeypatch.setattr(fq, "_run", lambda *a: pytest.fail("the library was called"))
    t, host = Made("cuda"), Made("cpu")
    names = {norm_fwd: ("x", "weight", "bias", "y", "mean", "rstd"),
             norm_bwd: ("dy", "x", "weight", "mean", "rstd", "dx", "dweight", "dbias"),
             product: ("xq", "s_x", "wq", "s_w", "y", "bias", "residual", "z"),
             act_bwd: ("dy", "z", "dz", "dbias"), norm: ("norm", "grads"),
             clip: ("norm", "grads", "out")}
    for call, args in names.items():
        for name in args:
            seen = {}
            with monkeypatch.context() as m:
                for f in ("layer_norm_fwd", "layer_norm_bwd", "melded_linear_fwd_act",
                          "linear_act_bwd", "grad_norm", "grad_clip"):
                    m.setattr(fq, f, lambda *a, **k: seen.update(k))
                call(t)
            v = seen[name]
            v = [v[0].cpu(), *v[1:]] if isinstance(v, list) else v.cpu()
            with pytest.raises(fq.FalqError, match="GPU|cuda"):
                call(t, **{name: v})
