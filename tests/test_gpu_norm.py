"""The root-mean-square norm on the GPU against its 64-bit form.

Tolerances.  u is half a step of the result's type (finfo.eps / 2), e = 2^-24
half a step of fp32; every sum of `cols` squares or products is at most 32 terms
in a lane, then 6 and 16 additions: 54 e relative to the sum of magnitudes, 64 e
with the quotient.
  h         one fp32 sum and one rounding: equal.
  r         (64 e / 2) for the sum under the root, the root and the quotient: 36 e.
  y         r and two products: 38 e |y| + u |y| (1 + 2^-20), plus half the smallest step.
  operand   of fp32 tensors: byte for byte what the quantiser makes of y.  Of
            16-bit ones: half a step of the code, 2^-4 or 2^-3 of the value (below
            the normals half the smallest step times the scale), with 38 e on
            top; exponents equal unless the block's maximum lies within 2^-16 of
            a border.
  dx        n and g one product each; the mean 64 e A, A the mean of |g n|;
            r (4 |g| + |n| (66 A + 4 |mean|)) e + 3 (|dres| + |dx|) e + u |dx|.
  dweight   n and product, 3 rows in a lane, 7 of a workgroup, 12 and 64 workgroups: 80 e
            sum |dy n| + e (|addend| + |dw|).
"""
import linear_forms as F
import numpy as np
import pytest
import train_forms as T

from communication_compressed_optimizer_elt_amd import binding as L

pytestmark = pytest.mark.gpu
E = 2.0**-24
DT = ["float32", "float16", "bfloat16"]


@pytest.fixture(scope="module")
def torch():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    L.lib()
    return torch


def host(t):
    return t.detach().double().cpu().numpy()


def normal(torch, seed, *shape, std=1.0, dtype="float32"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(getattr(torch, dtype)).cuda()


def half_step(torch, dtype):
    f = torch.finfo(getattr(torch, dtype))
    return f.eps / 2, f.tiny * f.eps / 2


def operand(torch, rows, cols):
    return torch.full((L.demo_block_layout(rows, cols)["total_bytes"],), 0xA5, dtype=torch.uint8, device="cuda")


def check_y(torch, y, want, dtype):
    u, low = half_step(torch, dtype)
    assert (np.abs(host(y) - want) <= (38 * E + u * (1 + 2.0**-20)) * np.abs(want) + low).all()


def check_operand(buf, want, fmt):
    """An operand of values that are known up to 38 e."""
    codes, e, clean = F.unpack(buf.cpu().numpy(), *want.shape, fmt)
    assert clean
    cols = want.shape[1]
    full = np.zeros((want.shape[0], -(-cols // 128) * 128))
    full[:, :cols] = np.abs(want)
    most = full.reshape(want.shape[0], -1, 128).max(2)
    lo = F.quantize(np.maximum(full * (1 - 2.0**-16), 0), fmt, 0)[1]
    hi = F.quantize(full * (1 + 2.0**-16), fmt, 0)[1]
    assert ((lo <= e) & (e <= hi)).all() and most.shape == e.shape
    digits, low = F.FORMATS[fmt][1:]
    wide = np.repeat(e, 128, 1)[:, :cols]
    bound = np.maximum(np.abs(want) * 2.0 ** -(digits + 1) * (1 + 2.0**-12), np.ldexp(0.5, low - digits + wide)) + 38 * E * np.abs(want)
    assert (np.abs(F.value(codes, e) - want) <= bound).all()


SHAPES = [(1, 1), (1, 2048), (3, 7), (130, 64), (5, 513), (64, 512), (2, 1000), (129, 1024), (2100, 1024), (2051, 2048),
          (2049, 1536), (16, 2049), (7, 4096), (6, 5000), (5, 8192), (3, 8200), (2, 16384), (1, 16383)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(torch, rows, cols, dtype, residual):
    x = normal(torch, rows + cols, rows, cols, dtype=dtype)
    res = normal(torch, rows, rows, cols, std=3.0, dtype=dtype) if residual else None
    w = normal(torch, cols, cols, std=0.5) + 1
    h, y = torch.full_like(x, 9.0), torch.full_like(x, 9.0)
    r = torch.full((rows,), 9.0, device="cuda")
    fmt = (rows + cols) % 2
    q, qt = operand(torch, rows, cols), operand(torch, cols, rows)
    L.demo_rms_norm(L.Norm(eps=1e-5, fmt=fmt), x, w, y=y, residual=res, h=h, rstd=r, operand=q, operand_t=qt)
    want_h = x if res is None else (x.float() + res.float()).to(x.dtype)
    assert torch.equal(h, want_h)
    want_r, want = T.norm(host(want_h), host(w), 1e-5)
    assert (np.abs(host(r) - want_r) <= 36 * E * want_r).all()
    check_y(torch, y, want, dtype)
    check_operand(q, want, fmt)
    check_operand(qt, want.T, fmt)
    if dtype == "float32":
        a, b = operand(torch, rows, cols), operand(torch, cols, rows)
        L.demo_block_quantize(L.Block(fmt=fmt), y, a, b)
        for got, same, (m, n) in ((q, a, (rows, cols)), (qt, b, (cols, rows))):
            for g, s in zip(F.unpack(got.cpu().numpy(), m, n, fmt), F.unpack(same.cpu().numpy(), m, n, fmt)):
                assert np.array_equal(g, s)
    # one output at a time gives the same
    for kw in (dict(y=torch.empty_like(y)), dict(rstd=torch.empty_like(r)), dict(operand=operand(torch, rows, cols)),
               dict(h=torch.empty_like(h))):
        L.demo_rms_norm(L.Norm(eps=1e-5, fmt=fmt), x, w, residual=res, **kw)
        (name, t), = kw.items()
        if name == "operand":
            assert all(np.array_equal(a, b) for a, b in zip(F.unpack(t.cpu().numpy(), rows, cols, fmt), F.unpack(q.cpu().numpy(), rows, cols, fmt)))
        else:
            assert torch.equal(t, {"y": y, "rstd": r, "h": h}[name])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("cols,pitch,at", [(200, 256, 0), (200, 301, 1), (2048, 2304, 128), (33, 40, 3)])
def test_norm_slices(torch, dtype, cols, pitch, at):
    """Column slices of wider matrices, aligned and not; what lies between the rows stays."""
    rows = 140
    wide = [normal(torch, 7 + i, rows, pitch, dtype=dtype) for i in range(4)]
    x, res, h, y = (t[:, at: at + cols] for t in wide)
    before = [t.clone() for t in wide]
    w, r = normal(torch, 3, cols) + 1, torch.empty(rows, device="cuda")
    q, qt = operand(torch, rows, cols), operand(torch, cols, rows)
    L.demo_rms_norm(L.Norm(), x, w, y=y, residual=res, h=h, rstd=r, operand=q, operand_t=qt)
    want_h = (x.float() + res.float()).to(x.dtype)
    assert torch.equal(h, want_h)
    _, want = T.norm(host(want_h), host(w), 1e-6)
    check_y(torch, y, want, dtype)
    check_operand(q, want, 0)
    check_operand(qt, want.T, 0)
    for t, b in zip(wide, before):
        t[:, at: at + cols] = 0
        b[:, at: at + cols] = 0
        assert torch.equal(t, b)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,cols", [(3, 2048), (2500, 600), (4, 5000)])
def test_norm_in_place(torch, dtype, rows, cols):
    x, res = normal(torch, 1, rows, cols, dtype=dtype), normal(torch, 2, rows, cols, dtype=dtype)
    w, cfg = normal(torch, 3, cols), L.Norm()
    h, y = torch.empty_like(x), torch.empty_like(x)
    L.demo_rms_norm(cfg, x, w, y=y, residual=res, h=h)
    a, b = x.clone(), res.clone()
    L.demo_rms_norm(cfg, a, w, y=a, residual=b, h=b)
    assert torch.equal(a, y) and torch.equal(b, h)
    a, b = x.clone(), torch.empty_like(x)
    L.demo_rms_norm(cfg, a, w, y=b, residual=res, h=a)
    assert torch.equal(a, h) and torch.equal(b, y)


def test_norm_of_odd_rows(torch):
    """Rows of zeros, infinities, NaN, subnormals and huge values, beside one that stays what it was."""
    cols = 640
    x = normal(torch, 1, 8, cols)
    w = normal(torch, 2, cols) + 2
    x[1], x[2, 5], x[3, 600] = 0, float("inf"), float("nan")
    x[4] = 1e-42
    x[5] = 1e18  # 640 * 1e36 = 6.4e38: the sum of its squares passes fp32's 3.4e38
    x[6] = 2e19  # each square does
    x[7, 130:200] = 0
    y, r = torch.empty_like(x), torch.empty(8, device="cuda")
    q, qt = operand(torch, 8, cols), operand(torch, cols, 8)
    L.demo_rms_norm(L.Norm(eps=1e-6), x, w, y=y, rstd=r, operand=q, operand_t=qt)
    assert not y[1].any() and abs(float(r[1]) - 1000.0) < 1e-3
    assert float(r[2]) == 0 and torch.isnan(y[2, 5]) and not y[2, 6:].any()
    assert torch.isnan(r[3]) and torch.isnan(y[3]).all()
    assert torch.isfinite(y[4]).all()
    assert not r[5:7].any() and not y[5:7].any()
    check_y(torch, y[7:], T.norm(host(x[7:]), host(w), 1e-6)[1], "float32")
    a, b = operand(torch, 8, cols), operand(torch, cols, 8)
    L.demo_block_quantize(L.Block(), y, a, b)
    for got, same, (m, n) in ((q, a, (8, cols)), (qt, b, (cols, 8))):
        for g, s in zip(F.unpack(got.cpu().numpy(), m, n, 0), F.unpack(same.cpu().numpy(), m, n, 0)):
            assert np.array_equal(g, s, equal_nan=True)
    x[5] = 7e17  # 640 * 4.9e35 = 3.1e38
    L.demo_rms_norm(L.Norm(eps=1e-6), x, w, y=y)
    check_y(torch, y[5:6], T.norm(host(x[5:6]), host(w), 1e-6)[1], "float32")
    L.demo_rms_norm(L.Norm(eps=0.0), x[:2].contiguous(), w, y=y[:2])
    assert torch.isnan(y[1]).all() and torch.isfinite(y[0]).all()


def check_backward(torch, dx, dw, dy, h, w, r, dres, addend, dtype):
    zero = 0.0 if dres is None else host(dres)
    want, want_w, a, s = T.norm_backward(host(dy), host(h), host(w), host(r), zero)
    n, g = host(h) * host(r)[:, None], host(dy) * host(w)
    mean = (g * n).mean(1, keepdims=True)
    u, low = half_step(torch, dtype)
    bound = E * (host(r)[:, None] * (4 * np.abs(g) + np.abs(n) * (66 * a + 4 * np.abs(mean))) + 3 * (np.abs(zero) + np.abs(want)))
    assert (np.abs(host(dx) - want) <= bound + u * (1 + 2.0**-20) * np.abs(want) + low).all()
    if dw is not None:
        add = 0.0 if addend is None else host(addend)
        assert (np.abs(host(dw) - add - want_w) <= E * (80 * s + np.abs(add) + np.abs(add + want_w))).all()


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_backward(torch, rows, cols, dtype, residual):
    h, dy = normal(torch, rows + cols, rows, cols, std=2.0, dtype=dtype), normal(torch, 5, rows, cols, dtype=dtype)
    dres = normal(torch, 6, rows, cols, dtype=dtype) if residual else None
    w, r = normal(torch, cols, cols) + 1, torch.empty(rows, device="cuda")
    cfg = L.Norm(eps=1e-5)
    L.demo_rms_norm(cfg, h, w, rstd=r)
    work = torch.empty(L.demo_rms_norm_workspace(cfg, rows, cols), dtype=torch.uint8, device="cuda")
    dx, dw = torch.full_like(h, 9.0), torch.full((cols,), 9.0, device="cuda")
    L.demo_rms_norm_backward(cfg, dy, h, w, r, dx, dresidual=dres, dweight=dw, workspace=work)
    check_backward(torch, dx, dw, dy, h, w, r, dres, None, dtype)
    grad = normal(torch, 8, cols, std=5.0)
    acc, other = grad.clone(), torch.empty_like(grad)
    L.demo_rms_norm_backward(cfg, dy, h, w, r, dx, dresidual=dres, dweight=acc, addend=acc, workspace=work)
    L.demo_rms_norm_backward(cfg, dy, h, w, r, dx, dresidual=dres, dweight=other, addend=grad, workspace=work)
    assert torch.equal(acc, other)  # and the order of sums is fixed
    check_backward(torch, dx, acc, dy, h, w, r, dres, grad, dtype)
    alone = torch.empty_like(dx)
    L.demo_rms_norm_backward(cfg, dy, h, w, r, alone, dresidual=dres)
    assert torch.equal(alone, dx)
    for name in ("dy", "h") + (("dres",) if residual else ()):  # in place
        t = {"dy": dy.clone(), "h": h.clone(), "dres": None if dres is None else dres.clone()}
        L.demo_rms_norm_backward(cfg, t["dy"], t["h"], w, r, t[name], dresidual=t["dres"])
        assert torch.equal(t[name], dx)


def test_norm_backward_slices(torch):
    rows, cols = 300, 333
    wide = [normal(torch, i, rows, 400, dtype="bfloat16") for i in range(4)]
    dy, h, dres, dx = (t[:, 5: 5 + cols] for t in wide)
    before = wide[3].clone()
    w, r = normal(torch, 9, cols), torch.empty(rows, device="cuda")
    L.demo_rms_norm(L.Norm(), h, w, rstd=r)
    L.demo_rms_norm_backward(L.Norm(), dy, h, w, r, dx, dresidual=dres)
    check_backward(torch, dx, None, dy, h, w, r, dres, None, "bfloat16")
    wide[3][:, 5: 5 + cols] = 0
    before[:, 5: 5 + cols] = 0
    assert torch.equal(wide[3], before)


def test_norm_gradient_by_differences(torch):
    """Central differences of sum(dy y) + sum(dres h) on the GPU.  They are off
    by 38 e sum |dy y| over the step, and by what the formula's own differences
    are off in 64 bits (which is the truncation)."""
    rows, cols, step = 3, 72, 2.0**-5
    x, res = normal(torch, 1, rows, cols), normal(torch, 2, rows, cols)
    dy, dres, w = normal(torch, 3, rows, cols), normal(torch, 4, rows, cols), normal(torch, 5, cols) + 1
    x, res = (torch.round(t * 256) / 256 for t in (x, res))  # x + res and the steps are exact
    cfg = L.Norm(eps=1e-3)
    y, h, r = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")

    def loss(x, w):
        L.demo_rms_norm(cfg, x, w, y=y, residual=res, h=h)
        return float((host(dy) * host(y)).sum() + (host(dres) * host(h)).sum()), np.abs(host(dy) * host(y)).sum()

    def loss64(x, w):
        h = host(x) + host(res)
        return (host(dy) * T.norm(h, host(w), float(np.float32(1e-3)))[1]).sum() + (host(dres) * h).sum()

    L.demo_rms_norm(cfg, x, w, y=y, residual=res, h=h, rstd=r)
    keep = h.clone()
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    work = torch.empty(L.demo_rms_norm_workspace(cfg, rows, cols), dtype=torch.uint8, device="cuda")
    L.demo_rms_norm_backward(cfg, dy, keep, w, r, dx, dresidual=dres, dweight=dw, workspace=work)
    r64 = T.norm(host(keep), host(w), float(np.float32(1e-3)))[0]
    dx64, dw64, _, _ = T.norm_backward(host(dy), host(keep), host(w), r64, host(dres))
    for i, j in ((0, 0), (1, 7), (2, 71), (0, 40), (1, 63)):
        e = torch.zeros_like(x)
        e[i, j] = step
        (up, a), (down, b) = loss(x + e, w), loss(x - e, w)
        slack = 38 * E * (a + b) / (2 * step) + abs((loss64(x + e, w) - loss64(x - e, w)) / (2 * step) - dx64[i, j])
        assert abs((up - down) / (2 * step) - float(dx[i, j])) <= slack + 200 * E * np.abs(dx64).max()
        e = torch.zeros_like(w)
        e[j] = step
        (up, a), (down, b) = loss(x, w + e), loss(x, w - e)
        assert abs((up - down) / (2 * step) - float(dw[j])) <= 40 * E * (a + b) / (2 * step) + 80 * E * np.abs(dw64).max()


@pytest.mark.parametrize("rows,cols", [(3, 1), (3, 70), (5, 2044), (3, 4100), (130, 200)])
def test_padding_of_nan_rows(torch, rows, cols):
    """Codes behind the last column and the last row are 0 beside NaN, infinities and negative weights too."""
    x = normal(torch, 1, rows, cols)
    x[1], x[rows - 1, 0] = float("nan"), float("inf")
    q, qt, r = operand(torch, rows, cols), operand(torch, cols, rows), torch.empty(rows, device="cuda")
    L.demo_rms_norm(L.Norm(), x, -1 - normal(torch, 2, cols).abs(), rstd=r, operand=q, operand_t=qt)
    codes, _, clean = F.unpack(q.cpu().numpy(), rows, cols, 0)
    turned, _, clean_t = F.unpack(qt.cpu().numpy(), cols, rows, 0)
    assert clean and clean_t
    assert np.isnan(codes[1]).all() and np.array_equal(np.isnan(turned), np.isnan(codes).T)
