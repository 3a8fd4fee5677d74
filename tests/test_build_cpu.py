"""The kernels compile without warnings: one that the compiler prints is a
promise it does not make (a reserved register among what a statement clobbers)
or code that does not do what it says."""
import os
import subprocess

import pytest

from communication_compressed_optimizer_elt_amd import build

# one instantiation of every kernel of the linear layer
KERNELS = """
#include "product_big.hpp"
#include "quantize.hpp"
using namespace demo;
template __global__ void demo::product_kernel<0, 0, false, 64, 64, 2, 2>(ProductArgs);
template __global__ void demo::product_kernel<0, 1, true, 128, 128, 2, 2>(ProductArgs);
template __global__ void demo::product_shared_kernel<0, 1>(ProductArgs);
template __global__ void demo::product_few_kernel<0, 0, false, 8>(ProductArgs);
template __global__ void demo::product_rows_kernel<0, 0, 1>(ProductArgs);
template __global__ void demo::product_big_kernel<0, 0>(ProductArgs);
template __global__ void demo::product_big_wide_kernel<0, 0>(ProductArgs);
template __global__ void demo::quantize_kernel<bf16_t, 0, false, true, true>(QuantArgs);
template __global__ void demo::quantize_kernel<float, 0, true, false, false>(QuantArgs);
template __global__ void demo::dropout_kernel<float, true>(DropoutArgs);
"""


@pytest.fixture(scope="module")
def warnings(tmp_path_factory):
    """The compiler's warnings about these kernels, for the GPU and for the host."""
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc here")
    src = tmp_path_factory.mktemp("kernels") / "kernels.hip"
    src.write_text(KERNELS)
    flags = [f for f in build.FLAGS if f != "-shared"] + ["-I", build.CSRC, "-I", os.path.join(build.ROOT, "include")]
    said = []
    for way in (["-c", "--offload-device-only", "-o", os.fspath(src) + ".o"], ["-fsyntax-only", "--offload-host-only"]):
        res = subprocess.run([build.HIPCC, *flags, "-Wno-unused-command-line-argument", *way, os.fspath(src)],
                             capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-4000:]
        said += [line for line in res.stderr.splitlines() if "warning: " in line]
    return said


def test_no_reserved_register_is_clobbered(warnings):
    assert not [w for w in warnings if "reserved register" in w][:3]


def test_no_access_past_an_array(warnings):
    assert not [w for w in warnings if "array index" in w][:3]


def test_no_warning_at_all(warnings):
    assert not warnings[:3]
