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

# Sources with matrix instructions in inline assembly, of which the compiler knows
# neither what they wait for nor which registers they keep: every build reads the
# assembly that became the library.  The second entry is a kernel that holds its sums in a0 to
# a255 by name, and the number of its instantiations.
INLINE_PRODUCTS = {"linear.hip": None, "mx.hip": ("mx_stream_kernel", 6)}


def build(verbose: bool = False) -> str:
    subprocess.check_call([sys.executable, os.path.join(CSRC, "gen_dct_consts.py")])
    with tempfile.TemporaryDirectory() as objects:
        compiled = [(s, os.path.join(objects, s + ".o")) for s in SOURCES]
        jobs = [[HIPCC, *(f for f in FLAGS if f != "-shared"), "-c", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                 *(["-save-temps=obj"] if s in INLINE_PRODUCTS else []), "-o", obj, os.path.join(CSRC, s)] for s, obj in compiled]
        with ThreadPoolExecutor(len(jobs)) as pool:
            done = list(pool.map(lambda cmd: _run(cmd, verbose), jobs))
        for source, named in INLINE_PRODUCTS.items():
            path, = glob.glob(os.path.join(objects, os.path.splitext(source)[0] + "-hip-amdgcn-*.s"))
            with open(path) as f:
                asm = f.read()
            check_waits(asm)
            if named:
                check_named_sums(asm, *named)
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


_NUMBER = r"(0x[0-9a-f]+|\d+)"


def _registers(text: str) -> set:
    """Vector registers named in operands: ('v' or 'a', number)."""
    out = {(k, int(n)) for k, n in re.findall(r"\b([va])(\d+)\b", text)}
    out |= {(k, int(n, 0)) for k, n in re.findall(rf"\b([va])\[{_NUMBER}\]", text)}
    for k, first, last in re.findall(rf"\b([va])\[{_NUMBER}:{_NUMBER}\]", text):
        out |= {(k, n) for n in range(int(first, 0), int(last, 0) + 1)}
    return out


# Wait states between a vector instruction and a matrix instruction that reads what it
# wrote, and between a matrix instruction and anything else that reads its sums: the
# most that the compiler keeps to for its own.
_OPERAND_WAIT, _RESULT_WAIT = 2, 18


def check_waits(asm: str) -> int:
    """Raises where a matrix instruction in inline assembly reads a register too soon
    after a vector instruction wrote it, or where its sums are read too soon, on any way
    through the code; returns how many of them there are."""
    wrong, count = [], 0
    for body in re.split(r"\n(?=_Z\w+:)", asm):
        code, labels, jumps, inline = [], {}, {}, False
        for line in body.split("\n"):
            if "#ASMSTART" in line or "#ASMEND" in line:
                inline = "#ASMSTART" in line
                continue
            text = line.split(";")[0].strip()
            label = re.match(r"(\.LBB\w+):", text)
            if label:
                labels[label[1]] = len(code)
            elif text and not text.endswith(":") and not text.startswith("."):
                op, _, rest = text.partition(" ")
                code.append((op, rest, inline))
                if op.startswith(("s_branch", "s_cbranch")):
                    jumps.setdefault(rest.strip(), []).append(len(code) - 1)
        if not any(inline and op.startswith("v_mfma") for op, _, inline in code):
            continue
        entries = {at: jumps.get(label, []) for label, at in labels.items()}

        def before(i, states):
            """Instructions at most `states` wait states in front of number i, on every way to it."""
            todo, seen = [(i, states)], {}
            while todo:
                at, left = todo.pop()
                ways = list(entries.get(at, []))
                if at and code[at - 1][0] not in ("s_branch", "s_endpgm"):
                    ways.append(at - 1)
                for j in ways:
                    if left <= 0 or seen.get(j, 0) >= left:
                        continue
                    seen[j] = left
                    op, rest, _ = code[j]
                    todo.append((j, left - (int(rest.split()[0], 0) + 1 if op == "s_nop" else 1)))
            return [code[j] for j in seen]

        for i, (op, rest, inline) in enumerate(code):
            parts = re.split(r",(?![^\[]*\])", rest)
            if op.startswith("v_mfma"):
                if inline:
                    count += 1
                    reads = _registers(",".join(parts[1:6]).split(" op_sel")[0])
                    wrong += [f"{o} {r}  ->  {op} {rest}" for o, r, _ in before(i, _OPERAND_WAIT)
                              if o.startswith("v_") and not o.startswith("v_mfma") and _registers(r.split(",")[0]) & reads]
            elif op.startswith(("v_", "ds_", "global_", "buffer_", "scratch_", "flat_")):
                sums = {x for x in _registers(",".join(parts[1:] if op.startswith("v_") else parts)) if x[0] == "a"}
                if sums:
                    wrong += [f"{o} {r}  ->  {op} {rest}" for o, r, asm_ in before(i, _RESULT_WAIT)
                              if asm_ and o.startswith("v_mfma") and _registers(r.split(",")[0]) & sums]
    if wrong:
        raise RuntimeError("operands or sums of matrix instructions are read too soon:\n" + "\n".join(wrong[:10]))
    return count


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
