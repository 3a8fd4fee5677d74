"""The build refuses code in which the compiler uses the registers that the 4-bit
product's largest kernel names for its sums: on assembly written here, and on the
kernel's own."""
import os
import subprocess

import pytest

from communication_compressed_optimizer_elt_amd import build

GOOD = """
_Z5otherv:
	v_accvgpr_write_b32 a3, v1
; ScratchSize: 16
_Z6kernelv:                             ; @_Z6kernelv
	v_add_u32_e32 v1, v2, v3
	;;#ASMSTART
	v_mfma_scale_f32_16x16x128_f8f6f4 a[0:3], v[0:3], v[4:7], a[0:3], v8, v9 op_sel:[0,0,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4
	;;#ASMEND
	s_mov_b32 m0, s2                        ; a comment on a3
	.amdhsa_next_free_vgpr a0
; ScratchSize: 0
"""


def test_checker():
    build.check_named_sums(GOOD, "6kernel", 1)
    for at, bad in (("	s_mov_b32 m0", "	v_accvgpr_write_b32 a17, v1"), ("	s_mov_b32 m0", "	ds_read_b128 a[4:7], v2"),
                    ("	s_mov_b32 m0", "	v_accvgpr_read_b32 v3, a255"), ("; ScratchSize: 0", "; ScratchSize: 8")):
        i = GOOD.rindex(at)
        with pytest.raises(RuntimeError, match="uses what 6kernel takes"):
            build.check_named_sums(GOOD[:i] + bad + "\n" + GOOD[i:], "6kernel", 1)
    for count in (0, 2):
        with pytest.raises(RuntimeError, match="instantiations"):
            build.check_named_sums(GOOD, "6kernel", count)


def test_kernel(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc here")
    src, asm = tmp_path / "stream.hip", tmp_path / "stream.s"
    src.write_text("""#include "mx_product.hpp"
template __global__ void demo::mx_stream_kernel<demo::bf16_t, true>(demo::ProductArgs);
template __global__ void demo::mx_stream_kernel<float, false>(demo::ProductArgs);
""")
    flags = [f for f in build.FLAGS if f != "-shared"] + ["-I", build.CSRC, "-I", os.path.join(build.ROOT, "include")]
    subprocess.run([build.HIPCC, *flags, "-S", "--offload-device-only", "-o", os.fspath(asm), os.fspath(src)], check=True,
                   capture_output=True)
    text = asm.read_text()
    build.check_named_sums(text, "mx_stream_kernel", 2)
    # its code is found by name: the tiles that keep their sums in variables do use these registers
    src.write_text("""#include "mx_product.hpp"
template __global__ void demo::mx_big_kernel<void>(demo::ProductArgs);
""")
    subprocess.run([build.HIPCC, *flags, "-S", "--offload-device-only", "-o", os.fspath(asm), os.fspath(src)], check=True,
                   capture_output=True)
    with pytest.raises(RuntimeError, match="uses what"):
        build.check_named_sums(asm.read_text(), "mx_big_kernel", 1)
