"""The rules that pick the kernels of the FP4 product and of the cross entropy,
compiled from their own headers for the host."""
import ctypes
import functools
import os
import subprocess
import tempfile

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "fp8_quantized_lora_amd", "csrc")

SOURCE = r"""
#include "cross_entropy_plan.hpp"
#include "mx_linear_plan.hpp"
using namespace falq;
// few, kind, split, kc
extern "C" void mx(int64_t M, int64_t N, int64_t K, int64_t* out) {
  const MxPlan p = mx_plan_of(M, N, K);
  out[0] = p.few;
  out[1] = p.kind;
  out[2] = p.split;
  out[3] = p.kc;
}
// the forward's kernel, G's (of the first piece), dx's, pieces, splits, strips
extern "C" void loss(int64_t T, int64_t d, int64_t V, int64_t* out) {
  const int64_t n = strip_of(T);
  const BwdPlan p = bwd_plan(n, d, V, 1);
  const int64_t ld = up(std::min(p.width, V), 64);
  out[0] = loss_kind(n, V, d);
  out[1] = grad_kind(n, ld, d);
  out[2] = p.kind;
  out[3] = ceil_div64(V, p.width);
  out[4] = p.splits;
  out[5] = ceil_div64(T, kStrip);
}
"""

MX_KINDS = ("256x128", "128", "64", "32x64")
LOSS_KINDS = ("256", "128", "64", "32x64")
GRAD_KINDS = ("256", "256x128", "192x128", "128", "64", "32x64")
DX_KINDS = ("256", "256x128", "128", "64", "32x64")


@functools.lru_cache(maxsize=1)
def _lib():
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", f"-I{CSRC}", src, "-o", so],
                       check=True)
        return ctypes.CDLL(so)


def _call(f, *sizes):
    out = (ctypes.c_int64 * 6)()
    f(*(ctypes.c_int64(s) for s in sizes), out)
    return list(out)


def mx(T, d_in, d_out):
    few, kind, split, _, _, _ = _call(_lib().mx, T, d_out, d_in // 2)
    return f"few{few}" if few else "split" if split > 1 else MX_KINDS[kind]


def loss(T, d, V):
    """(forward's kernel, G's, dx's, "*" behind those split, pieces, strips)"""
    f, g, x, pieces, splits, strips = _call(_lib().loss, T, d, V)
    return (LOSS_KINDS[f], GRAD_KINDS[g], DX_KINDS[x] + "*" * (splits > 1), pieces, strips)
