"""The norm, gradient clipping and the 4-bit layer without a GPU: layouts,
refusals, and the tests' own plain forms against torch's.  No call here
launches."""
import ctypes
import os

import numpy as np
import pytest
import torch
import train_forms as T

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
    assert ctypes.sizeof(L.demo_norm_cfg) == ctypes.sizeof(L.demo_mx_cfg) == 16
    assert ctypes.sizeof(L.demo_tensor) == 24 and L.demo_tensor.dtype.offset == 16


# --------------------------------------------------------------- plain forms --

def test_plain_backward_is_torch_s():
    g = torch.Generator().manual_seed(1)
    h, w, dy, dres = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((5, 33), (33,), (5, 33), (5, 33)))
    h.requires_grad_(True), w.requires_grad_(True)
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 0.1) * w
    ((y * dy).sum() + (h * dres).sum()).backward()
    r, plain = T.norm(h.detach().numpy(), w.detach().numpy(), 0.1)
    dx, dw, _, _ = T.norm_backward(dy.numpy(), h.detach().numpy(), w.detach().numpy(), r, dres.numpy())
    assert np.allclose(plain, y.detach().numpy(), rtol=1e-12, atol=0)
    assert np.allclose(dx, h.grad.numpy(), rtol=1e-10, atol=1e-13) and np.allclose(dw, w.grad.numpy(), rtol=1e-10, atol=1e-13)


def test_plain_rounding_goes_to_the_nearest_code():
    v = np.linspace(-6, 6, 4801)
    got, near = T.mx_round(v), np.abs(np.abs(v)[:, None] - T.GRID)
    assert np.array_equal(np.abs(np.abs(v) - np.abs(got)), near.min(1))
    halves = {0.25: 0, 0.75: 1, 1.25: 1, 1.75: 2, 2.5: 2, 3.5: 4, 5: 4}  # to the even code
    assert [float(x) for x in T.mx_round(np.array(list(halves)))] == list(map(float, halves.values()))


def test_plain_scales_are_the_smallest():
    x = np.exp2(np.linspace(-140, 120, 3000))[:, None] * np.ones((1, 32))
    codes, e = T.mx_quantize(x, 0)
    assert (np.abs(codes) <= 6).all()
    fits = x[:, :1] <= 6 * np.exp2(e - 1.0)
    assert not (fits & (e > -127)).any() and (e >= -127).all()


def test_plain_packing_round_trip():
    g = np.random.default_rng(2)
    for rows, cols in ((1, 1), (3, 31), (5, 257), (33, 512)):
        codes, e = T.mx_quantize(g.normal(size=(rows, cols)), rows % 2)
        back, be, clean = T.mx_unpack(T.mx_pack(codes, e), rows, cols)
        assert clean and np.array_equal(back, codes) and np.array_equal(be, e)


# ---------------------------------------------------------------------- norm --

NORM = L.Norm().c(L.DTYPE_BF16)


def norm_call(cfg=NORM, rows=130, cols=200, x=FAR, ld_x=200, res=2 * FAR, ld_res=200, w=3 * FAR, h=4 * FAR, ld_h=200,
              y=5 * FAR, ld_y=200, rstd=6 * FAR, q=7 * FAR, qt=8 * FAR):
    return L.raw_rms_norm(cfg, rows, cols, x, ld_x, res, ld_res, w, h, ld_h, y, ld_y, rstd, q, qt)


@pytest.mark.parametrize("kw,code", [
    (dict(cfg=None), L.EINVAL), (dict(cfg=L.Norm(abi_version=2).c()), L.EABI), (dict(cfg=L.Norm().c(3)), L.EINVAL),
    (dict(cfg=L.Norm(fmt=2).c()), L.EINVAL), (dict(cfg=L.Norm(eps=-1e-6).c()), L.EINVAL),
    (dict(cfg=L.Norm(eps=float("nan")).c()), L.EINVAL), (dict(cfg=L.Norm(eps=float("inf")).c()), L.EINVAL),
    (dict(rows=0), L.EINVAL), (dict(cols=0), L.EINVAL), (dict(rows=2**30 + 1), L.EINVAL),
    (dict(cols=16385, ld_x=16385, ld_res=16385, ld_h=16385, ld_y=16385), L.EUNSUPPORTED),
    (dict(ld_x=199), L.EINVAL), (dict(ld_res=199), L.EINVAL), (dict(ld_h=199), L.EINVAL), (dict(ld_y=199), L.EINVAL),
    (dict(ld_x=2**36), L.EINVAL), (dict(x=None), L.EINVAL), (dict(w=None), L.EINVAL),
    (dict(h=None, y=None, rstd=None, q=None, qt=None), L.EINVAL),
    (dict(rstd=None), L.EINVAL),  # the transposed operand is made from r
    (dict(h=None), L.EINVAL),  # and from h
    (dict(x=FAR + 1), L.EALIGN), (dict(res=2 * FAR + 1), L.EALIGN), (dict(w=3 * FAR + 2), L.EALIGN), (dict(h=4 * FAR + 1), L.EALIGN),
    (dict(y=5 * FAR + 1), L.EALIGN), (dict(rstd=6 * FAR + 2), L.EALIGN), (dict(q=7 * FAR + 8), L.EALIGN), (dict(qt=8 * FAR + 4), L.EALIGN),
    (dict(h=FAR + 400), L.EINVAL), (dict(y=4 * FAR), L.EINVAL), (dict(rstd=3 * FAR), L.EINVAL), (dict(q=FAR), L.EINVAL),
    (dict(qt=7 * FAR + 1024), L.EINVAL), (dict(h=3 * FAR), L.EINVAL), (dict(h=FAR, ld_h=256), L.EINVAL),
    (dict(res=None, h=None, y=FAR), L.EINVAL),  # x is read again
    (dict(q=4 * FAR + 256), L.EINVAL), (dict(x=6 * FAR), L.EINVAL),
])
def test_norm_refusals(kw, code):
    assert norm_call(**kw) == code


def back_call(cfg=NORM, rows=130, cols=200, dy=FAR, ld_dy=200, h=2 * FAR, ld_h=200, w=3 * FAR, rstd=4 * FAR, dres=5 * FAR,
              ld_dres=200, dx=6 * FAR, ld_dx=200, dw=7 * FAR, addend=8 * FAR, work=9 * FAR, have=L.BLOCK_MAX_WORKSPACE):
    return L.raw_rms_norm_backward(cfg, rows, cols, dy, ld_dy, h, ld_h, w, rstd, dres, ld_dres, dx, ld_dx, dw, addend, work, have)


@pytest.mark.parametrize("kw,code", [
    (dict(cfg=None), L.EINVAL), (dict(cfg=L.Norm(abi_version=2).c()), L.EABI), (dict(rows=0), L.EINVAL),
    (dict(cols=16385, ld_dy=16385, ld_h=16385, ld_dres=16385, ld_dx=16385), L.EUNSUPPORTED), (dict(ld_dy=199), L.EINVAL),
    (dict(ld_h=199), L.EINVAL), (dict(ld_dres=1), L.EINVAL), (dict(ld_dx=199), L.EINVAL), (dict(dy=None), L.EINVAL),
    (dict(h=None), L.EINVAL), (dict(w=None), L.EINVAL), (dict(rstd=None), L.EINVAL), (dict(dx=None), L.EINVAL),
    (dict(dw=None), L.EINVAL),  # an addend of nothing
    (dict(work=None), L.EINVAL), (dict(have=100), L.EINVAL), (dict(work=9 * FAR + 8), L.EALIGN), (dict(dy=FAR + 1), L.EALIGN),
    (dict(dw=7 * FAR + 2), L.EALIGN), (dict(addend=8 * FAR + 1), L.EALIGN), (dict(rstd=4 * FAR + 2), L.EALIGN),
    (dict(dx=FAR + 2), L.EINVAL), (dict(dx=FAR, ld_dx=208), L.EINVAL), (dict(dx=3 * FAR), L.EINVAL), (dict(dw=3 * FAR), L.EINVAL),
    (dict(dw=6 * FAR), L.EINVAL), (dict(dw=FAR), L.EINVAL), (dict(addend=7 * FAR + 4), L.EINVAL), (dict(dx=8 * FAR), L.EINVAL),
    (dict(work=FAR), L.EINVAL), (dict(work=8 * FAR), L.EINVAL), (dict(work=7 * FAR - 256), L.EINVAL), (dict(dw=4 * FAR + 16), L.EINVAL),
])
def test_norm_backward_refusals(kw, code):
    assert back_call(**kw) == code


def test_norm_workspace():
    for rows, cols in ((1, 1), (16384, 2048), (2**20, 16384), (3, 16384)):
        rc, need = L.raw_rms_norm_workspace(NORM, rows, cols)
        assert rc == L.OK and 0 < need <= L.BLOCK_MAX_WORKSPACE
    assert L.raw_rms_norm_workspace(NORM, 1, 16385)[0] == L.EUNSUPPORTED
    assert L.raw_rms_norm_workspace(None, 1, 1)[0] == L.EINVAL
    assert L.lib().demo_rms_norm_workspace(ctypes.byref(NORM), 1, 1, None) == L.EINVAL


# ------------------------------------------------------------------ gradient --

def test_grad_refusals():
    big = 1 << 20  # elements: more than one workgroup's
    good = L.raw_tensors((FAR, big, 0), (2 * FAR, 100, 2))
    ws = dict(workspace=4 * FAR, workspace_bytes=L.BLOCK_MAX_WORKSPACE)
    for bad, code in ((L.raw_tensors((FAR, 100, 3)), L.EINVAL), (L.raw_tensors((FAR, 100, 0, 1)), L.EINVAL),
                      (L.raw_tensors((None, 100, 0)), L.EINVAL), (L.raw_tensors((FAR, 2**36 + 1, 0)), L.EINVAL),
                      (L.raw_tensors((FAR + 2, 100, 0)), L.EALIGN), (L.raw_tensors((FAR + 1, 100, 1)), L.EALIGN)):
        assert L.raw_grad_norm(1, bad, 3 * FAR, **ws) == code
        assert L.raw_grad_workspace(1, bad)[0] == code
        assert L.raw_grad_clip(1, bad, None, 3 * FAR, 1.0) == code
        assert L.raw_grad_clip(1, L.raw_tensors((5 * FAR, 100, 1)), bad, 3 * FAR, 1.0) in (code, L.EINVAL)
    assert L.raw_grad_norm(L.MAX_TENSORS + 1, good, 3 * FAR, **ws) == L.EINVAL
    assert L.raw_grad_norm(2, None, 3 * FAR, **ws) == L.EINVAL
    assert L.raw_grad_norm(2, good, None, **ws) == L.EINVAL
    assert L.raw_grad_norm(2, good, 3 * FAR + 4, **ws) == L.EALIGN
    assert L.raw_grad_norm(2, good, 3 * FAR, 4 * FAR + 8, 1 << 20) == L.EALIGN
    assert L.raw_grad_norm(2, good, 3 * FAR) == L.EINVAL  # no workspace
    need = L.raw_grad_workspace(2, good)[1]
    assert 0 < need <= L.BLOCK_MAX_WORKSPACE
    assert L.raw_grad_norm(2, good, 3 * FAR, 4 * FAR, need - 1) == L.EINVAL
    assert L.raw_grad_norm(2, good, FAR, **ws) == L.EINVAL  # the sum inside a tensor
    assert L.raw_grad_norm(2, good, 3 * FAR, 2 * FAR, 1 << 20) == L.EINVAL  # the workspace over one
    assert L.raw_grad_norm(2, good, 4 * FAR + 8, **ws) == L.EINVAL  # the sum inside the workspace
    assert L.lib().demo_grad_workspace(2, good, None) == L.EINVAL


def test_grad_workspace_sizes():
    assert L.raw_grad_workspace(0, None) == (L.OK, 0)
    assert L.raw_grad_workspace(2, L.raw_tensors((FAR, 1000, 0), (None, 0, 1))) == (L.OK, 0)
    many = L.raw_tensors(*[(FAR + (i << 30), 1 << 26, 0) for i in range(2000)])
    rc, need = L.raw_grad_workspace(2000, many)
    assert rc == L.OK and 0 < need <= L.BLOCK_MAX_WORKSPACE
    most = (L.demo_tensor * L.MAX_TENSORS)(*[L.demo_tensor(FAR, 1 << 36, 0, 0)] * L.MAX_TENSORS)
    rc, need = L.raw_grad_workspace(L.MAX_TENSORS, most)
    assert rc == L.OK and 0 < need <= L.BLOCK_MAX_WORKSPACE


def test_clip_refusals():
    def call(src, dst=None, sumsq=9 * FAR, limit=1.0, norm=8 * FAR):
        return L.raw_grad_clip(len(src), L.raw_tensors(*src), None if dst is None else L.raw_tensors(*dst), sumsq, limit, norm)

    one = [(FAR, 100, 2), (2 * FAR, 50, 0)]
    assert call(one, sumsq=None) == call(one, limit=-1.0) == call(one, limit=float("nan")) == L.EINVAL
    assert call(one, sumsq=9 * FAR + 4) == call(one, norm=8 * FAR + 2) == L.EALIGN
    assert call(one, [(3 * FAR, 100, 2), (4 * FAR, 51, 0)]) == L.EINVAL  # another size
    assert call(one, [(3 * FAR, 100, 1), (4 * FAR, 50, 0)]) == L.EINVAL  # neither src's type nor fp32
    assert call(one, [(3 * FAR, 100, 2), (4 * FAR, 50, 2)]) == L.EINVAL
    assert call(one, [(FAR, 100, 0), (4 * FAR, 50, 0)]) == L.EINVAL  # in place with another type
    assert call(one, [(FAR + 2, 100, 2), (4 * FAR, 50, 0)]) == L.EINVAL  # beside its own place
    assert call(one, [(2 * FAR, 100, 2), (4 * FAR, 50, 0)]) == L.EINVAL  # over another source
    assert call(one, [(3 * FAR, 100, 2), (3 * FAR + 64, 50, 0)]) == L.EINVAL  # over one another
    assert call([one[0], one[0]]) == L.EINVAL  # the same tensor twice in place
    assert call(one, norm=FAR) == call(one, sumsq=FAR) == call(one, norm=9 * FAR) == call(one, norm=9 * FAR + 4) == L.EINVAL


def test_tensors_refuse_host_tensors():
    with pytest.raises(ValueError, match="device tensor"):
        L.Tensors([torch.zeros(4)])
    with pytest.raises(ValueError, match="device tensor"):
        L.demo_grad_norm([], torch.zeros(1, dtype=torch.float64))
    assert len(L.Tensors([])) == 0 and L.demo_grad_workspace([]) == 0


# ------------------------------------------------------------------ 4 bits --

@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 255), (128, 256), (2561, 768), (7, 513), (5, 2048)])
def test_mx_layout(rows, cols):
    got = L.demo_mx_layout(rows, cols)
    assert tuple(got[k] for k in ("pitch", "scale_off", "scale_pitch", "total_bytes")) == T.mx_layout(rows, cols)


def test_mx_layout_refusals():
    for rows, cols in ((0, 1), (1, 0), (2**30 + 1, 1), (1, 2**30 + 1), (2**20, 2**17)):
        assert L.raw_mx_layout(rows, cols)[0] == L.EINVAL
    assert L.raw_mx_layout(2**30, 64)[0] == L.OK
    assert L.lib().demo_mx_layout(1, 1, None) == L.EINVAL


def test_mx_quantize_refusals():
    def call(cfg=L.Mx().c(L.DTYPE_BF16), rows=130, cols=200, src=FAR, ld=200, drop=None, q=2 * FAR, qt=3 * FAR):
        return L.raw_mx_quantize(cfg, rows, cols, src, ld, drop, q, qt)

    assert call(None) == call(L.Mx(tile=2).c(0)) == call(L.Mx(reserved=1).c(0)) == call(L.Mx().c(3)) == L.EINVAL
    assert call(L.Mx(abi_version=7).c(0)) == L.EABI
    assert call(drop=L.Dropout(p=2.0)) == call(drop=L.Dropout(chunk_offset=2**59)) == L.EINVAL
    assert call(rows=0) == call(cols=0) == call(ld=199) == call(src=None) == call(ld=2**36) == L.EINVAL
    assert call(rows=2**30 + 1) == call(q=None, qt=None) == L.EINVAL
    assert call(src=FAR + 1) == call(q=2 * FAR + 8) == call(qt=3 * FAR + 4) == L.EALIGN
    assert call(q=FAR + 1024) == call(qt=FAR - 1024) == call(qt=2 * FAR + 256) == L.EINVAL  # overlaps


def test_mx_dequantize_refusals():
    def call(cfg=L.Mx().c(L.DTYPE_BF16), rows=130, cols=200, q=FAR, dst=2 * FAR, ld=200):
        return L.raw_mx_dequantize(cfg, rows, cols, q, dst, ld)

    assert call(None) == call(L.Mx(tile=1).c(0)) == call(L.Mx().c(3)) == L.EINVAL
    assert call(L.Mx(abi_version=7).c(0)) == L.EABI
    assert call(rows=0) == call(ld=199) == call(q=None) == call(dst=None) == call(dst=FAR + 512) == L.EINVAL
    assert call(q=FAR + 8) == call(dst=2 * FAR + 1) == L.EALIGN


def test_mx_matmul_refusals():
    def call(cfg=L.Mx().c(L.DTYPE_BF16), m=64, n=96, k=300, a=FAR, b=2 * FAR, c=3 * FAR, ldc=96, **kw):
        return L.raw_mx_matmul(cfg, m, n, k, a, b, c, ldc, **kw)

    assert call(None) == call(L.Mx(tile=1).c()) == call(L.Mx().c(3)) == call(L.Mx(reserved=5).c()) == L.EINVAL
    assert call(L.Mx(abi_version=3).c()) == L.EABI
    assert call(m=0) == call(n=0) == call(k=0) == call(ldc=95) == L.EINVAL
    assert call(a=None) == call(b=None) == call(c=None) == L.EINVAL
    assert call(ldc=2**36) == call(addend=4 * FAR, ld_addend=2**36) == call(dropout=L.Dropout(site=1 << 24)) == L.EINVAL
    assert call(k=L.BLOCK_MAX_K + 1) == L.EUNSUPPORTED
    assert call(m=2**30 + 1) == L.EINVAL
    assert call(a=FAR + 8) == call(b=2 * FAR + 4) == call(c=3 * FAR + 1) == L.EALIGN
    assert call(addend=4 * FAR + 1, ld_addend=96) == call(workspace=5 * FAR + 8) == L.EALIGN
    assert call(addend=4 * FAR, ld_addend=95) == L.EINVAL
    assert call(c=FAR + 256) == call(c=2 * FAR) == L.EINVAL  # c over an operand
    assert call(addend=3 * FAR + 64, ld_addend=96) == L.EINVAL  # neither c itself nor clear of it
    assert call(addend=3 * FAR, ld_addend=128) == L.EINVAL  # c with another pitch


def test_mx_workspace_sizes():
    some = 0
    for m, n, k in ((1, 2048, 8192), (2304, 768, 2561), (4096, 8192, 2048), (768, 768, 1 << 22), (64, 64, 1 << 22), (17, 16384, 16384),
                    (64, 64, 16384), (2048, 2048, 16384)):
        rc, need = L.raw_mx_workspace(L.Mx().c(), m, n, k)
        assert rc == L.OK and need <= L.BLOCK_MAX_WORKSPACE
        if need:
            some += 1
            args = (L.Mx().c(L.DTYPE_F32), m, n, k, FAR, 2 * FAR, 3 * FAR, n)
            assert L.raw_mx_matmul(*args) == L.EINVAL
            assert L.raw_mx_matmul(*args, workspace=4 * FAR, workspace_bytes=need - 1) == L.EINVAL
            assert L.raw_mx_matmul(*args, workspace=3 * FAR + 256, workspace_bytes=need) == L.EINVAL  # over c
    assert some
    assert L.raw_mx_workspace(L.Mx().c(), 1, 1, 0)[0] == L.EINVAL
    assert L.raw_mx_workspace(None, 1, 1, 1)[0] == L.EINVAL


def test_binding_refuses_host_tensors():
    x, u = torch.zeros(16, 128), torch.zeros(1 << 16, dtype=torch.uint8)
    w = torch.ones(128)
    for call in (lambda: L.demo_rms_norm(L.Norm(), x, w, y=x.clone()),
                 lambda: L.demo_rms_norm_backward(L.Norm(), x, x, w, torch.ones(16), x.clone()),
                 lambda: L.demo_mx_quantize(L.Mx(), x, u), lambda: L.demo_mx_dequantize(u, x),
                 lambda: L.demo_mx_matmul(L.Mx(), 16, 128, 16, u, u, x)):
        with pytest.raises(ValueError, match="device tensor"):
            call()


def test_mx_quantize_refuses_grids_that_are_too_large():
    """2^30 rows of one column are 2^23 squares, and as many beside them whose codes are padding."""
    for rows, cols in ((2**30, 1), (2**30 - 127, 1)):
        assert L.raw_mx_quantize(L.Mx().c(L.DTYPE_BF16), rows, cols, FAR, cols, None, 2**50, None) == L.EUNSUPPORTED
