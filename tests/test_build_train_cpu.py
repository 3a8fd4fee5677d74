"""The kernels of the norm, of the gradient's clipping and of the 4-bit layer
compile without warnings, as the linear layer's do."""
import os
import subprocess

import pytest

from communication_compressed_optimizer_elt_amd import build

# one instantiation of every kernel
KERNELS = """
#include "grad.hpp"
#include "mx_product.hpp"
#include "mx_quantize.hpp"
#include "norm.hpp"
using namespace demo;
template __global__ void demo::norm_kernel<bf16_t, 4, 1, true>(NormArgs);
template __global__ void demo::norm_kernel<float, 16, 2, false>(NormArgs);
template __global__ void demo::norm_turn_kernel<f16_t, 0, true>(NormTurnArgs);
template __global__ void demo::norm_back_kernel<bf16_t, 2, 1, true>(NormBackArgs);
template __global__ void demo::norm_back_kernel<float, 16, 2, false>(NormBackArgs);
template __global__ void demo::grad_norm_kernel<4>(GradArgs);
template __global__ void demo::grad_scale_kernel<true>(GradArgs);
template __global__ void demo::mx_quantize_kernel<bf16_t, true, true, true>(MxArgs);
template __global__ void demo::mx_quantize_kernel<float, false, false, false>(MxArgs);
template __global__ void demo::mx_values_kernel<f16_t, true>(MxValuesArgs);
template __global__ void demo::mx_kernel<64, 64, 2, 2, 4>(ProductArgs);
template __global__ void demo::mx_kernel<128, 128, 2, 2, 2>(ProductArgs);
template __global__ void demo::mx_big_kernel<void>(ProductArgs);
template __global__ void demo::mx_stream_kernel<bf16_t, false>(ProductArgs);
template __global__ void demo::mx_stream_kernel<float, true>(ProductArgs);
template __global__ void demo::mx_few_kernel<4>(ProductArgs);
template __global__ void demo::mx_rows_kernel<2>(ProductArgs);
"""


def test_no_warning(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc here")
    src = tmp_path / "kernels.hip"
    src.write_text(KERNELS)
    flags = [f for f in build.FLAGS if f != "-shared"] + ["-I", build.CSRC, "-I", os.path.join(build.ROOT, "include")]
    for way in (["-c", "--offload-device-only", "-o", os.fspath(src) + ".o"], ["-fsyntax-only", "--offload-host-only"]):
        res = subprocess.run([build.HIPCC, *flags, "-Wno-unused-command-line-argument", *way, os.fspath(src)],
                             capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-4000:]
        assert not [line for line in res.stderr.splitlines() if "warning: " in line][:3]
