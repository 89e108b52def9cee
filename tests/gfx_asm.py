"""The built library's GPU code as instructions, for tests of what inline asm
leaves to its writer: the compiler puts no wait states between its own
instructions and those of an asm statement."""
import functools
import os
import re
import shutil
import subprocess
import tempfile
from typing import NamedTuple, Optional

import fp8_quantized_lora_amd as fq


class Ins(NamedTuple):
    op: str
    args: tuple                   # operands, destination first
    at: int                       # address
    target: Optional[int]         # a branch's

    def __str__(self):
        return f"{self.at:#x}: {self.op} {', '.join(self.args)}"

    @property
    def states(self):
        """Wait states that the instruction stands for."""
        return int(self.args[0], 0) + 1 if self.op == "s_nop" else 1


def objdump():
    """The disassembler beside hipcc's compiler (None: not installed)."""
    hipcc = shutil.which("hipcc")
    roots = ([os.path.dirname(os.path.dirname(os.path.realpath(hipcc)))] if hipcc else [])
    for r in [*roots, "/opt/rocm"]:
        for sub in ("llvm/bin", "lib/llvm/bin", "bin"):
            p = os.path.join(r, sub, "llvm-objdump")
            if os.path.exists(p):
                return p
    return shutil.which("llvm-objdump")


def registers(text, kinds="va"):
    """The registers an operand names, as (kind, number)."""
    out = set()
    for m in re.finditer(rf"\b([{kinds}])(?:\[(\d+):(\d+)\]|(\d+)\b)", text):
        lo, hi = (m[2], m[3]) if m[2] else (m[4], m[4])
        out |= {(m[1], i) for i in range(int(lo), int(hi) + 1)}
    return out


def parse(text):
    """{function: [Ins]} of a disassembly."""
    out, cur, base = {}, None, 0
    for line in text.splitlines():
        m = re.match(r"^([0-9a-f]+) <(.*)>:", line)
        if m:
            base, cur = int(m[1], 16), out.setdefault(m[2], [])
            continue
        m = re.match(r"^\t(\S+)\s*(.*?)\s*// ([0-9A-F]+):(.*)", line)
        if not m or cur is None:
            continue
        args = tuple(a.strip() for a in re.split(r",\s*(?![^\[]*\])", m[2]) if a.strip())
        to = re.search(r"<[^>+]*(?:\+0x([0-9a-f]+))?>", m[4])
        target = base + int(to[1] or "0", 16) if to and "branch" in m[1] else None
        cur.append(Ins(m[1], args, int(m[3], 16), target))
    return out


@functools.lru_cache(maxsize=1)
def functions():
    """{function: [Ins]} of every kernel in the built library."""
    out = {}
    with tempfile.TemporaryDirectory() as d:
        lib = shutil.copy(fq.LIB_PATH, d)
        subprocess.run([objdump(), "--offloading", lib], cwd=d, check=True, capture_output=True)
        for f in sorted(os.listdir(d)):
            if "gfx950" in f:
                r = subprocess.run([objdump(), "-d", os.path.join(d, f)], check=True,
                                   capture_output=True, text=True)
                out.update(parse(r.stdout))
    return out


def before(ins, k, states):
    """The instructions that precede number k by fewer than `states` wait states,
    along the listing."""
    j, w = k - 1, 0
    while j >= 0 and w < states:
        yield ins[j]
        w += ins[j].states
        j -= 1


def after(ins, k, states):
    """(instruction, wait states since) for what may follow number k by fewer than
    `states` wait states, along every path; send(True) ends a path."""
    at = {i.at: n for n, i in enumerate(ins)}
    seen, todo = {}, [(k + 1, 0)]
    while todo:
        j, w = todo.pop()
        if j >= len(ins) or w >= states or seen.get(j, states) <= w:
            continue
        seen[j] = w
        i = ins[j]
        if (yield i, w):
            yield
            continue
        if i.op == "s_endpgm":
            continue
        if i.target is not None:
            todo.append((at[i.target], w + 1))
            if i.op == "s_branch":
                continue
        todo.append((j + 1, w + i.states))
