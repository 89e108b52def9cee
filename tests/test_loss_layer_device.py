"""LinearCrossEntropy on a device that is not the current one: every call of its methods is
made with the layer's device current (on the host, with the calls recorded)."""
import contextlib

import torch

import fp8_quantized_lora_amd as fq
from fp8_quantized_lora_amd import step

CALLS = ("fp8_quantize", "linear_cross_entropy_fwd", "linear_cross_entropy_bwd")


class Loss:
    def __init__(self, device):
        self.device = torch.device(device)


def record(monkeypatch, current):
    seen, now = [], [current]

    @contextlib.contextmanager
    def device(dev):
        was, now[0] = now[0], dev.index
        yield
        now[0] = was
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    for name in CALLS:
        monkeypatch.setattr(step, name, lambda *a, name=name, **k: seen.append((name, now[0])))
    monkeypatch.setattr(step, "_arg", lambda *a: None)
    monkeypatch.setattr(step, "_device", lambda t, name: t.device.index)
    monkeypatch.setattr(step, "_stream_of", lambda dev, stream: 0)
    monkeypatch.setattr(step, "_on_stream", lambda *a: contextlib.nullcontext())
    return seen, now


def test_methods_run_on_the_layers_device(monkeypatch):
    for current in (0, 1):
        head = fq.LinearCrossEntropy(50, 32, 4, device="cpu")
        head.loss = Loss("cuda:1")
        seen, now = record(monkeypatch, current)
        head.init_state(None)
        head.forward(None, torch.zeros(4, dtype=torch.int64))
        head.backward(None)
        assert seen == [(n, 1) for n in ("fp8_quantize", "fp8_quantize",
                                         "linear_cross_entropy_fwd", "linear_cross_entropy_bwd")]
        assert now == [current]
