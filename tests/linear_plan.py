"""The rule that picks the FP8 product's kernel, compiled from its own header for
the host."""
import ctypes
import functools
import os
import subprocess
import tempfile
from typing import NamedTuple

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "fp8_quantized_lora_amd", "csrc")

SOURCE = r"""
#include "linear_act_plan.hpp"
using namespace falq;
// few, kind, split, kc, and the workgroups and threads of each of its first launch
extern "C" void plan(int64_t M, int64_t N, int64_t K, int64_t* out) {
  const Plan p = plan_of(M, N, K);
  out[0] = p.few;
  out[1] = p.kind;
  out[2] = p.split;
  out[3] = p.kc;
  if (p.few) {
    out[4] = (N + 15) / 16;
    out[5] = kFewWaves[p.few] * 64;
  } else {
    const TileKind k = p.split > 1 ? k128w8 : p.kind;
    out[4] = tiles_of(k, M, N) * p.split;
    out[5] = k == k128w8 || k == k128x192w8 ? 512 : 256;
  }
}
extern "C" int kinds() { return kTileKinds; }
"""

KINDS = ("256x320", "256", "256x128", "128x256", "192x128", "128x192w8", "128", "128w8", "64",
         "32x64")


class Plan(NamedTuple):
    how: str                      # "few1", "few2", "split" or a tile kind
    split: int
    groups: int
    threads: int


@functools.lru_cache(maxsize=1)
def _lib():
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", f"-I{CSRC}", src, "-o", so],
                       check=True)
        lib = ctypes.CDLL(so)
    assert lib.kinds() == len(KINDS)
    return lib


def plan(T, d_in, d_out):
    out = (ctypes.c_int64 * 6)()
    i64 = ctypes.c_int64
    _lib().plan(i64(T), i64(d_out), i64(d_in), out)
    how = f"few{out[0]}" if out[0] else "split" if out[2] > 1 else KINDS[out[1]]
    return Plan(how, out[2], out[4], out[5])
