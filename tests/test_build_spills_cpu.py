"""What the norm's backward pass keeps in scratch memory: nothing up to 8192 columns, at
most twelve registers of a lane beyond, as its comment says."""
import os
import re
import subprocess

import pytest

from communication_compressed_optimizer_elt_amd import build

KERNELS = """#include "norm.hpp"
using namespace demo;
template __global__ void demo::norm_back_kernel<float, 1, 1, true>(NormBackArgs);
template __global__ void demo::norm_back_kernel<bf16_t, 4, 1, true>(NormBackArgs);
template __global__ void demo::norm_back_kernel<bf16_t, 8, 1, false>(NormBackArgs);
template __global__ void demo::norm_back_kernel<float, 16, 1, true>(NormBackArgs);
template __global__ void demo::norm_back_kernel<float, 16, 1, false>(NormBackArgs);
template __global__ void demo::norm_back_kernel<float, 16, 2, true>(NormBackArgs);
template __global__ void demo::norm_back_kernel<f16_t, 16, 2, true>(NormBackArgs);
template __global__ void demo::norm_back_kernel<bf16_t, 16, 2, true>(NormBackArgs);
template __global__ void demo::norm_back_kernel<float, 16, 2, false>(NormBackArgs);
template __global__ void demo::norm_back_kernel<f16_t, 16, 2, false>(NormBackArgs);
template __global__ void demo::norm_back_kernel<bf16_t, 16, 2, false>(NormBackArgs);
"""


def test_spills(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc here")
    src = tmp_path / "back.hip"
    src.write_text(KERNELS)
    flags = [f for f in build.FLAGS if f != "-shared"] + ["-I", build.CSRC, "-I", os.path.join(build.ROOT, "include")]
    res = subprocess.run([build.HIPCC, *flags, "-c", "--offload-device-only", "-Rpass-analysis=kernel-resource-usage", "-o",
                          os.fspath(src) + ".o", os.fspath(src)], check=True, capture_output=True, text=True)
    spills = dict(re.findall(r"Function Name: (\S+norm_back_kernel\S+).*?VGPRs Spill: (\d+)", res.stderr, re.S))
    assert len(spills) == 11
    for name, count in spills.items():
        most = (12 if "Lb0E" in name else 5) if "Li16ELi2E" in name else 0
        assert int(count) <= most, (name, count)
