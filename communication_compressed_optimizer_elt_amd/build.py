"""Build libdemo.so (HIP, gfx950) in-tree with hipcc."""
from __future__ import annotations

import os
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


def build(verbose: bool = False) -> str:
    subprocess.check_call([sys.executable, os.path.join(CSRC, "gen_dct_consts.py")])
    with tempfile.TemporaryDirectory() as objects:
        compiled = [(s, os.path.join(objects, s + ".o")) for s in SOURCES]
        jobs = [[HIPCC, *(f for f in FLAGS if f != "-shared"), "-c", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                 "-o", obj, os.path.join(CSRC, s)] for s, obj in compiled]
        with ThreadPoolExecutor(len(jobs)) as pool:
            done = list(pool.map(lambda cmd: _run(cmd, verbose), jobs))
        tmp = LIB + ".tmp"
        done.append(_run([HIPCC, *LINK_FLAGS, "-o", tmp, *(obj for _, obj in compiled)], verbose))
    # the host's pass does not know the GPU's feature, and says so every time
    said = [line for text in done for line in text.splitlines(True)
            if "'-packed-fp32-ops' is not a recognized feature" not in line]
    sys.stderr.write("".join(said))
    os.replace(tmp, LIB)
    return LIB


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
