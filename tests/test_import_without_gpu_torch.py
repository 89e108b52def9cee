"""The package imports, and its host-side calls run, on a torch that was built
without a GPU (its private accessors of streams and devices are not there)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import fp8_quantized_lora_amd as fq
assert fq.version() and fq.layer_norm_bwd_workspace_bytes(4096, 64) > 0
m = fq.MeldedLinear(64, 32, 4, 16, device="cpu", bias=True, act="gelu")
try:
    x = torch.zeros(4, 64)
    fq.layer_norm_fwd(x, None, None, x.clone())
except fq.FalqError as e:
    assert "GPU" in str(e), e
else:
    raise AssertionError("a CPU tensor was accepted")
print("imported")
"""


def test_import():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr[-2000:]
