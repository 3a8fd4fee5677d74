"""Build libdemo.so (HIP, gfx950) in-tree with hipcc."""
from __future__ import annotations

import glob
import os
import re
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libdemo.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # no packed fp32 instructions anywhere in the library
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
]
LINK_FLAGS = ["--offload-arch=gfx950", "-fPIC", "-shared"]


SOURCES = ["demo.hip", "linear.hip", "grad.hip", "norm.hip", "mx.hip"]

# The kernel whose inline assembly holds its sums in a0 to a255 by name from one
# statement to the next, which no constraint tells the compiler: every build reads the
# assembly that became the library and refuses one that uses such a register elsewhere.
NAMED_SUMS = {"mx.hip": ("mx_stream_kernel", 6)}  # its instantiations


def build(verbose: bool = False) -> str:
    subprocess.check_call([sys.executable, os.path.join(CSRC, "gen_dct_consts.py")])
    with tempfile.TemporaryDirectory() as objects:
        compiled = [(s, os.path.join(objects, s + ".o")) for s in SOURCES]
        jobs = [[HIPCC, *(f for f in FLAGS if f != "-shared"), "-c", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                 *(["-save-temps=obj"] if s in NAMED_SUMS else []), "-o", obj, os.path.join(CSRC, s)] for s, obj in compiled]
        with ThreadPoolExecutor(len(jobs)) as pool:
            done = list(pool.map(lambda cmd: _run(cmd, verbose), jobs))
        for source, (kernel, count) in NAMED_SUMS.items():
            asm, = glob.glob(os.path.join(objects, os.path.splitext(source)[0] + "-hip-amdgcn-*.s"))
            with open(asm) as f:
                check_named_sums(f.read(), kernel, count)
        tmp = LIB + ".tmp"
        done.append(_run([HIPCC, *LINK_FLAGS, "-o", tmp, *(obj for _, obj in compiled)], verbose))
    # the host's pass does not know the GPU's feature, and says so every time
    said = [line for text in done for line in text.splitlines(True)
            if "'-packed-fp32-ops' is not a recognized feature" not in line]
    sys.stderr.write("".join(said))
    os.replace(tmp, LIB)
    return LIB


def check_named_sums(asm: str, kernel: str, count: int) -> None:
    """Raises where one of the `count` instantiations of `kernel` in this assembly names
    an accumulator register outside its inline assembly, or keeps anything in memory of
    its own (a spill, which could go to such a register next time)."""
    found, name, inline, wrong = set(), None, False, []
    for line in asm.splitlines():
        if "#ASMSTART" in line or "#ASMEND" in line:
            inline = "#ASMSTART" in line
            continue
        label = re.match(r"(_Z\w+):", line)
        if label:
            name = label[1] if kernel in label[1] else None
            found |= {name} - {None}
        if name is None:
            continue
        scratch = re.match(r"; ScratchSize: (\d+)", line)
        code = line.split(";")[0].strip()
        if scratch and int(scratch[1]) or (not inline and not code.startswith(".") and re.search(r"\ba(\d|\[)", code)):
            wrong.append(f"{name}: {line.strip()}")
    if len(found) != count:
        raise RuntimeError(f"{len(found)} instantiations of {kernel} in its assembly, not {count}")
    if wrong:
        raise RuntimeError(f"the compiler uses what {kernel} takes for its sums:\n" + "\n".join(wrong[:10]))


def _run(cmd: list, verbose: bool) -> str:
    """What the compiler says on stderr."""
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("hipcc failed to build libdemo.so")
    return res.stderr


if __name__ == "__main__":
    print(build(verbose=True))
