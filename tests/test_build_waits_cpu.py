"""The build refuses matrix instructions in inline assembly that read an operand, or whose
sums are read, before the wait states are over: on assembly written here, and on the kernels
that have such instructions."""
import os
import subprocess

import pytest

from communication_compressed_optimizer_elt_amd import build

MFMA = "	;;#ASMSTART\n	v_mfma_f32_32x32x16_bf16 a[0:15], v[50:53], v[58:61], a[0:15]\n	;;#ASMEND\n"
HEAD, END = "\n_Z1kv:                                  ; @_Z1kv\n", "	s_endpgm\n.Lfunc_end0:\n"


def kernel(*lines):
    return HEAD + "".join(x if x.startswith("	;;") else f"	{x}\n" if not x.startswith(".") else x + "\n" for x in lines) + END


@pytest.mark.parametrize("lines", [
    ("v_mov_b32_e32 v61, v1", "s_nop 1", MFMA),
    ("v_mov_b32_e32 v61, v1", "s_nop 0", "s_mov_b32 s1, s2", MFMA),
    ("v_mov_b32_e32 v62, v1", MFMA),  # another register
    ("ds_read_b128 v[58:61], v1", MFMA),  # no vector instruction
    (MFMA, MFMA),  # the same sums again
    (MFMA, "s_nop 15", "s_nop 1", "v_accvgpr_read_b32 v1, a0"),
    (MFMA, "v_accvgpr_read_b32 v1, a16"),
    ("v_mov_b32_e32 v61, v1", "s_branch .LBB0_2", ".LBB0_1:", MFMA, ".LBB0_2:", "s_nop 0"),  # not on a way to it
])
def test_good(lines):
    assert build.check_waits(kernel(*lines)) == "".join(lines).count("v_mfma")


@pytest.mark.parametrize("lines", [
    ("v_mov_b32_e32 v61, v1", MFMA),
    ("v_mov_b32_e32 v50, v1", "s_nop 0", MFMA),
    ("v_cvt_scalef32_pk_bf16_fp8 v61, v39, v94 op_sel:[1,0,0]", "s_cmp_ge_u32 s47, s50", MFMA),
    ("v_accvgpr_write_b32 a15, v1", MFMA),
    ("v_pk_mov_b32 v[60:61], v[2:3], v[4:5]", "s_waitcnt lgkmcnt(0)", MFMA),
    (MFMA, "s_nop 15", "s_nop 0", "v_accvgpr_read_b32 v1, a0"),
    (MFMA, "ds_write_b128 v1, a[12:15]"),
    (MFMA, "v_accvgpr_read_b32 v1, a[0xf]"),
    (".LBB0_1:", MFMA, "s_nop 2", "v_mov_b32_e32 v61, v1", "s_cbranch_scc0 .LBB0_1"),  # round the loop
    ("v_mov_b32_e32 v61, v1", "s_branch .LBB0_2", ".LBB0_1:", "s_nop 1", ".LBB0_2:", MFMA),  # by the branch
])
def test_bad(lines):
    with pytest.raises(RuntimeError, match="too soon"):
        build.check_waits(kernel(*lines))


def test_the_compiler_s_own_are_its_own():
    assert build.check_waits(kernel("v_mov_b32_e32 v61, v1", "v_mfma_f32_32x32x16_bf16 a[0:15], v[50:53], v[58:61], a[0:15]")) == 0


@pytest.mark.parametrize("source,count", [
    ('#include "mx_product.hpp"\ntemplate __global__ void demo::mx_big_kernel<void>(demo::ProductArgs);\n', 512),
    ('#include "product_big.hpp"\ntemplate __global__ void demo::product_big_kernel<0, 1>(demo::ProductArgs);\n'
     'template __global__ void demo::product_big_wide_kernel<0, 1>(demo::ProductArgs);\n', 576),
])
def test_kernels(tmp_path, source, count):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc here")
    src, asm = tmp_path / "kernel.hip", tmp_path / "kernel.s"
    src.write_text(source)
    flags = [f for f in build.FLAGS if f != "-shared"] + ["-I", build.CSRC, "-I", os.path.join(build.ROOT, "include")]
    subprocess.run([build.HIPCC, *flags, "-S", "--offload-device-only", "-o", os.fspath(asm), os.fspath(src)], check=True,
                   capture_output=True)
    assert build.check_waits(asm.read_text()) == count
