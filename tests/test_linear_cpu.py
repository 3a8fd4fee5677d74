"""The low-precision linear layer without a GPU: layouts, refusals, and the
tests' own plain forms against torch's conversions.  No call here launches."""
import ctypes
import os
import subprocess
import sys

import linear_forms as F
import numpy as np
import pytest
import torch

from communication_compressed_optimizer_elt_amd import binding as L

A = 1 << 20  # fake, aligned addresses for calls that return before launching
FAR = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(L.LIB_PATH):
        from communication_compressed_optimizer_elt_amd import build

        build.build()
    return L.lib()


def test_struct_sizes():
    assert ctypes.sizeof(L.demo_dropout_cfg) == 40 and L.demo_dropout_cfg.seed.offset == 16
    assert ctypes.sizeof(L.demo_operand) == 32
    assert ctypes.sizeof(L.demo_block_cfg) == ctypes.sizeof(L.demo_product_cfg) == 16


def test_philox_known_answers():
    """The generator's published known answers (all zeros, all ones)."""
    assert [int(x) for x in F.philox(0, 0, 0, 0, 0, 0)] == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    f = 0xFFFFFFFF
    assert [int(x) for x in F.philox(f, f, f, f, f, f)] == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


@pytest.mark.parametrize("fmt,dtype", [(0, torch.float8_e4m3fn), (1, torch.float8_e5m2)])
def test_plain_codes_are_torch_s(fmt, dtype):
    every = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(F.decode_codes(every.numpy(), fmt), every.view(dtype).double().numpy(), equal_nan=True)
    x = torch.randn(5000, generator=torch.Generator().manual_seed(1)) * torch.logspace(-7, 2, 5000)
    assert np.array_equal(F.round_to(x.double().numpy(), fmt), x.to(dtype).double().numpy())


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 127), (128, 128), (2561, 768), (7, 129), (100352, 2048), (5, 513)])
def test_layout(rows, cols):
    got = L.demo_block_layout(rows, cols)
    assert tuple(got[k] for k in ("pitch", "scale_off", "scale_pitch", "total_bytes")) == F.layout(rows, cols)


def test_layout_refusals():
    for rows, cols in ((0, 1), (1, 0), (2**30 + 1, 1), (1, 2**30 + 1), (2**20, 2**17)):
        assert L.raw_block_layout(rows, cols)[0] == L.EINVAL
    assert L.raw_block_layout(2**30, 64)[0] == L.OK
    assert L.lib().demo_block_layout(1, 1, None) == L.EINVAL


@pytest.mark.parametrize("kw,code", [
    (dict(abi_version=2), L.EABI), (dict(p=-0.1), L.EINVAL), (dict(p=1.5), L.EINVAL), (dict(p=float("nan")), L.EINVAL),
    (dict(site=1 << 24), L.EINVAL), (dict(reserved=1), L.EINVAL), (dict(chunk_offset=2**59), L.EINVAL),
    (dict(chunk_offset=2**64 - 1), L.EINVAL),
])
def test_bad_dropouts(kw, code):
    d = L.Dropout(**kw)
    assert L.raw_dropout(d, L.DTYPE_F32, 64, A, None, 2 * A) == code
    assert L.raw_dropout_backward(d, L.DTYPE_F32, 64, A, 2 * A) == code
    q = L.Block().c(L.DTYPE_F32)
    assert L.raw_block_quantize(q, 8, 8, A, 8, d, 2 * A, None) == code
    p = L.Product().c()
    assert L.raw_block_matmul(p, 8, 8, 8, A, 2 * A, 3 * A, 8, dropout=d) == code


def test_dropout_refusals():
    d = L.Dropout()
    assert L.raw_dropout(None, 0, 64, A, None, 2 * A) == L.EINVAL
    for n in (0, 2**36 + 1):
        assert L.raw_dropout(d, 0, n, A, None, FAR) == L.EINVAL
    assert L.raw_dropout(d, 3, 64, A, None, 2 * A) == L.EINVAL
    assert L.raw_dropout(d, 0, 64, None, None, 2 * A) == L.EINVAL
    assert L.raw_dropout(d, 0, 64, A, None, None) == L.EINVAL
    assert L.raw_dropout(d, 0, 64, A + 4, None, 2 * A) == L.EALIGN
    assert L.raw_dropout(d, 0, 64, A, None, 2 * A + 8) == L.EALIGN
    assert L.raw_dropout(d, 0, 64, A, 3 * A + 2, 2 * A) == L.EALIGN
    assert L.raw_dropout(d, 0, 64, A, None, A + 128) == L.EINVAL  # y inside x
    assert L.raw_dropout(d, 0, 64, A, 2 * A + 16, 2 * A) == L.EINVAL  # residual overlaps y
    assert L.raw_dropout_backward(d, 1, 64, A, A + 112) == L.EINVAL


def test_quantize_refusals():
    def call(cfg=None, rows=130, cols=200, src=FAR, ld=200, q=2 * FAR, qt=3 * FAR):
        return L.raw_block_quantize(cfg or L.Block().c(L.DTYPE_BF16), rows, cols, src, ld, None, q, qt)

    assert L.raw_block_quantize(None, 130, 200, FAR, 200, None, 2 * FAR, None) == L.EINVAL
    assert call(L.Block(abi_version=7).c(0)) == L.EABI
    for bad in (L.Block(fmt=2).c(0), L.Block(tile=2).c(0), L.Block().c(3)):
        assert call(bad) == L.EINVAL
    assert call(rows=0) == call(cols=0) == call(ld=199) == call(src=None) == L.EINVAL
    assert call(ld=2**36) == L.EINVAL  # (rows - 1) ld past 2^40
    assert call(rows=2**30 + 1) == call(q=None, qt=None) == L.EINVAL
    assert call(src=FAR + 1) == call(q=2 * FAR + 8) == call(qt=3 * FAR + 4) == L.EALIGN
    assert call(q=FAR + 1024) == call(qt=FAR - 1024) == call(qt=2 * FAR + 256) == L.EINVAL  # overlaps


def test_matmul_refusals():
    def call(cfg=None, m=64, n=96, k=300, a=FAR, b=2 * FAR, c=3 * FAR, ldc=96, **kw):
        return L.raw_block_matmul(cfg or L.Product().c(L.DTYPE_BF16), m, n, k, a, b, c, ldc, **kw)

    assert L.raw_block_matmul(None, 64, 96, 300, FAR, 2 * FAR, 3 * FAR, 96) == L.EINVAL
    assert call(L.Product(abi_version=3).c()) == L.EABI
    for bad in (L.Product(fmt_a=2).c(), L.Product(fmt_b=9).c(), L.Product().c(3)):
        assert call(bad) == L.EINVAL
    assert call(m=0) == call(n=0) == call(k=0) == call(ldc=95) == L.EINVAL
    assert call(a=None) == call(b=None) == call(c=None) == L.EINVAL
    assert call(ldc=2**36) == call(addend=4 * FAR, ld_addend=2**36) == L.EINVAL  # (m - 1) ldc past 2^40
    assert call(k=L.BLOCK_MAX_K + 1) == L.EUNSUPPORTED
    assert call(m=2**30 + 1) == L.EINVAL
    assert call(a=FAR + 8) == call(b=2 * FAR + 4) == call(c=3 * FAR + 1) == L.EALIGN
    assert call(addend=4 * FAR + 1, ld_addend=96) == call(workspace=5 * FAR + 8) == L.EALIGN
    assert call(addend=4 * FAR, ld_addend=95) == L.EINVAL
    assert call(c=FAR + 256) == call(c=2 * FAR) == L.EINVAL  # c over an operand
    assert call(addend=3 * FAR + 64, ld_addend=96) == L.EINVAL  # neither c itself nor clear of it
    assert call(addend=3 * FAR, ld_addend=128) == L.EINVAL  # c with another pitch


def test_matmul_refuses_slices_of_one_matrix():
    """Columns 0..95 of a matrix of 192 as c, 96..191 as addend: their spans overlap."""
    args = (L.Product().c(L.DTYPE_F32), 64, 96, 300, FAR, 2 * FAR)
    assert L.raw_block_matmul(*args, 3 * FAR, 192, addend=3 * FAR + 4 * 96, ld_addend=192) == L.EINVAL
    assert L.raw_block_matmul(*args, 3 * FAR + 4 * 96, 192, addend=3 * FAR, ld_addend=192) == L.EINVAL


def test_workspace_sizes():
    for m, n, k in ((1, 2048, 8192), (2304, 768, 2561), (4096, 8192, 2048), (768, 768, 1 << 22), (64, 64, 1 << 22)):
        rc, need = L.raw_block_workspace(L.Product().c(), m, n, k)
        assert rc == L.OK and need <= L.BLOCK_MAX_WORKSPACE
        if need:
            args = (L.Product().c(L.DTYPE_F32), m, n, k, FAR, 2 * FAR, 3 * FAR, n)
            assert L.raw_block_matmul(*args) == L.EINVAL
            assert L.raw_block_matmul(*args, workspace=4 * FAR, workspace_bytes=need - 1) == L.EINVAL
            assert L.raw_block_matmul(*args, workspace=3 * FAR + 256, workspace_bytes=need) == L.EINVAL  # over c
    assert L.raw_block_workspace(L.Product().c(), 1, 1, 0)[0] == L.EINVAL
    assert L.raw_block_workspace(None, 1, 1, 1)[0] == L.EINVAL


def test_binding_refuses_host_tensors():
    x = torch.zeros(16, 128)
    u = torch.zeros(1 << 16, dtype=torch.uint8)
    for call in (lambda: L.demo_dropout(L.Dropout(), x, x.clone()), lambda: L.demo_dropout_backward(L.Dropout(), x, x),
                 lambda: L.demo_block_quantize(L.Block(), x, u), lambda: L.demo_block_matmul(L.Product(), 16, 128, 16, u, u, x)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(TypeError, match="float32, float16 or bfloat16"):
        L.demo_dropout(L.Dropout(), x.double(), x.double())


@pytest.mark.parametrize("call", ["demo_block_layout(3, 4)", "demo_abi_version()"])
def test_one_hip_runtime_whatever_comes_first(call):
    """A call that needs no GPU, before torch is imported: the library binds to
    torch's HIP runtime, not to a second one whose streams are others."""
    code = ("from communication_compressed_optimizer_elt_amd import binding as L\n"
            f"L.{call}\n"
            "import torch\n"
            "print(len({line.split()[-1] for line in open('/proc/self/maps') if 'libamdhip64' in line}))")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    assert res.stdout.split() == ["1"]
