"""The norm and its backward pass where a workgroup takes several rows one after
another, against 64 bits on the GPU and, bit for bit, against calls on so few rows
that each workgroup has one.

A launch has 2^20 workgroups of four rows up to 512 columns, 2^20 of one row up to
six waves' columns, 4096 up to 4096 columns, 512 beyond; the backward pass 512
workgroups of 8, 4, 2 or 1 rows at a time, 256 beyond 4096 columns.

Tolerances: test_gpu_norm's, u half a step of the type and e = 2^-24: 36 e for r, 38 e
and u for y, its bound for dx.  dweight: n and its product 2 e of |dy n|, a lane's rows
one e each, at most 7 additions in the workgroup, the rest in 64 bits and one rounding:
(p + 9) e sum |dy n| + e (|addend| + |dw|) with p rows a lane.
"""
import pytest

from communication_compressed_optimizer_elt_amd import binding as L

pytestmark = pytest.mark.gpu
E = 2.0**-24


@pytest.fixture(scope="module")
def torch():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    L.lib()
    return torch


def normal(torch, seed, *shape, std=1.0, dtype="float32"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(getattr(torch, dtype))


def rounding(torch, dtype):
    f = torch.finfo(getattr(torch, dtype))
    return f.eps / 2, f.tiny * f.eps / 2


def operand(torch, rows, cols):
    return torch.zeros(L.demo_block_layout(rows, cols)["total_bytes"], dtype=torch.uint8, device="cuda")


def parts(buf, rows, cols):
    """Codes and scale bytes of an operand, by rows."""
    o = L.demo_block_layout(rows, cols)
    codes = buf[: rows * o["pitch"]].view(rows, o["pitch"])
    return codes, buf[o["scale_off"]: o["scale_off"] + rows * o["scale_pitch"]].view(rows, o["scale_pitch"])


def check_rows(torch, x, res, w, h, y, r, dtype, eps):
    """h, r and y of some rows against 64 bits."""
    want_h = x if res is None else (x.float() + res.float()).to(x.dtype)
    assert torch.equal(h, want_h)
    v = want_h.double()
    want_r = 1 / ((v * v).mean(1) + eps).sqrt()
    assert ((r.double() - want_r).abs() <= 36 * E * want_r).all()
    want = v * want_r[:, None] * w.double()
    u, low = rounding(torch, dtype)
    assert ((y.double() - want).abs() <= (38 * E + u * (1 + 2.0**-20)) * want.abs() + low).all()


# rows, columns, rows of which each is a workgroup's only one
MANY = [(1100, 8200, 512), (1537, 16384, 512), (1100, 5000, 512), (1030, 6001, 512), (9000, 4096, 4096), (8300, 3100, 4096),
        (9000, 3999, 4096)]


@pytest.mark.parametrize("rows,cols,few", MANY)
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("residual", [False, True])
def test_rows_one_after_another(torch, rows, cols, few, dtype, residual):
    x = normal(torch, rows + cols, rows, cols, dtype=dtype)
    x *= 1 + torch.arange(rows, device="cuda")[:, None] % 5  # a row with another's statistics shows
    res = normal(torch, 2, rows, cols, std=3.0, dtype=dtype) if residual else None
    w = normal(torch, 3, cols, std=0.5) + 1
    h, y, r = torch.full_like(x, 9.0), torch.full_like(x, 9.0), torch.full((rows,), 9.0, device="cuda")
    q = operand(torch, rows, cols)
    cfg = L.Norm(eps=1e-5)
    L.demo_rms_norm(cfg, x, w, y=y, residual=res, h=h, rstd=r, operand=q)
    check_rows(torch, x, res, w, h, y, r, dtype, float(torch.tensor(1e-5)))
    if dtype == "float32":  # byte for byte what the quantiser makes of y
        same = operand(torch, rows, cols)
        L.demo_block_quantize(L.Block(), y, same)
        assert all(torch.equal(a, b) for a, b in zip(parts(q, rows, cols), parts(same, rows, cols)))
    codes, scales = parts(q, rows, cols)
    for i in range(0, rows, few):
        n = min(few, rows - i)
        s = slice(i, i + n)
        one = operand(torch, n, cols)
        oh, oy, orr = torch.empty_like(x[s]), torch.empty_like(x[s]), torch.empty(n, device="cuda")
        L.demo_rms_norm(cfg, x[s], w, y=oy, residual=None if res is None else res[s], h=oh, rstd=orr, operand=one)
        c, b = parts(one, n, cols)
        assert torch.equal(oh, h[s]) and torch.equal(oy, y[s]) and torch.equal(orr, r[s])
        assert torch.equal(c, codes[s]) and torch.equal(b, scales[s])
    a, b = x.clone(), torch.empty_like(x)  # in place: x is loaded ahead of what is written over it
    L.demo_rms_norm(cfg, a, w, y=b, residual=res, h=a)
    assert torch.equal(a, h) and torch.equal(b, y)
    if residual:
        a, b = x.clone(), res.clone()
        L.demo_rms_norm(cfg, a, w, y=a, residual=b, h=b)
        assert torch.equal(a, y) and torch.equal(b, h)


@pytest.mark.parametrize("rows,cols,dtype", [((2 << 22) + 5, 8, "float32"), ((1 << 22) + 3, 7, "bfloat16"),
                                             ((1 << 20) + 70, 520, "float32"), ((2 << 20) + 3, 513, "float16")])
def test_a_million_rows(torch, rows, cols, dtype):
    """Columns of few waves, whose grids hold a million workgroups."""
    x = normal(torch, 1, rows, cols, dtype=dtype)
    w = normal(torch, 3, cols, std=0.5) + 1
    y, r = torch.full_like(x, 9.0), torch.full((rows,), 9.0, device="cuda")
    q = operand(torch, rows, cols)
    L.demo_rms_norm(L.Norm(eps=1e-5), x, w, y=y, rstd=r, operand=q)
    eps, step = float(torch.tensor(1e-5)), 1 << 18
    for i in range(0, rows, step):
        s = slice(i, i + step)
        check_rows(torch, x[s], None, w, x[s], y[s], r[s], dtype, eps)
    codes, scales = parts(q, rows, cols)
    for i in (0, rows - 4099):  # the first rows, and the last ones, which are a workgroup's second or third
        s = slice(i, i + 4099)
        one = operand(torch, 4099, cols)
        L.demo_rms_norm(L.Norm(eps=1e-5), x[s], w, operand=one)
        c, b = parts(one, 4099, cols)
        assert torch.equal(c, codes[s]) and torch.equal(b, scales[s])
    a = x.clone()
    L.demo_rms_norm(L.Norm(eps=1e-5), a, w, y=a)
    assert torch.equal(a, y)


# rows, columns, rows a workgroup takes at a time, workgroups
BACK = [(13000, 500, 8, 512), (4200, 1000, 4, 512), (2500, 1536, 2, 512), (3100, 2047, 2, 512), (1100, 2100, 1, 512),
        (1600, 3100, 1, 512), (1100, 4096, 1, 512), (600, 5000, 1, 256), (600, 8192, 1, 256), (600, 8200, 1, 256), (600, 16384, 1, 256),
        (520, 16383, 1, 256)]


@pytest.mark.parametrize("rows,cols,each,grid", BACK)
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("residual", [False, True])
def test_backward_rows_one_after_another(torch, rows, cols, each, grid, dtype, residual):
    assert rows > each * grid
    h, dy = normal(torch, rows + cols, rows, cols, std=2.0, dtype=dtype), normal(torch, 5, rows, cols, dtype=dtype)
    dy *= 1 + torch.arange(rows, device="cuda")[:, None] % 5
    dres = normal(torch, 6, rows, cols, dtype=dtype) if residual else None
    w, r, add = normal(torch, cols, cols) + 1, torch.empty(rows, device="cuda"), normal(torch, 8, cols, std=5.0)
    cfg = L.Norm(eps=1e-5)
    L.demo_rms_norm(cfg, h, w, rstd=r)
    work = torch.empty(L.demo_rms_norm_workspace(cfg, rows, cols), dtype=torch.uint8, device="cuda")
    dx, dw = torch.full_like(h, 9.0), torch.full((cols,), 9.0, device="cuda")
    L.demo_rms_norm_backward(cfg, dy, h, w, r, dx, dresidual=dres, dweight=dw, addend=add, workspace=work)
    n, g = h.double() * r.double()[:, None], dy.double() * w.double()
    mean, a = (g * n).mean(1, keepdim=True), (g * n).abs().mean(1, keepdim=True)
    zero = torch.zeros((), device="cuda", dtype=torch.float64) if dres is None else dres.double()
    want = r.double()[:, None] * (g - n * mean) + zero
    u, low = rounding(torch, dtype)
    bound = E * (r.double()[:, None] * (4 * g.abs() + n.abs() * (66 * a + 4 * mean.abs())) + 3 * (zero.abs() + want.abs()))
    assert ((dx.double() - want).abs() <= bound + u * (1 + 2.0**-20) * want.abs() + low).all()
    check_dw(torch, dw, dy, h, r, add, -(-rows // (each * grid)))
    for i in range(0, rows, each * grid):
        s = slice(i, i + each * grid)
        one = torch.empty_like(dx[s])
        L.demo_rms_norm_backward(cfg, dy[s], h[s], w, r[s], one, dresidual=None if dres is None else dres[s])
        assert torch.equal(one, dx[s])
    for name in ("dy", "h") + (("dres",) if residual else ()):  # in place
        t = {"dy": dy.clone(), "h": h.clone(), "dres": None if dres is None else dres.clone()}
        L.demo_rms_norm_backward(cfg, t["dy"], t["h"], w, r, t[name], dresidual=t["dres"])
        assert torch.equal(t[name], dx)


def check_dw(torch, dw, dy, h, r, add, lane_rows):
    want, s = torch.zeros(dw.shape, dtype=torch.float64, device="cuda"), torch.zeros(dw.shape, dtype=torch.float64, device="cuda")
    for i in range(0, dy.shape[0], 1 << 18):
        t = dy[i: i + (1 << 18)].double() * (h[i: i + (1 << 18)].double() * r[i: i + (1 << 18)].double()[:, None])
        want += t.sum(0)
        s += t.abs().sum(0)
    want += add.double()
    assert ((dw.double() - want).abs() <= E * ((lane_rows + 9) * s + add.double().abs() + want.abs())).all()


@pytest.mark.parametrize("rows,cols,each", [(200_003, 300, 8), (1_000_001, 33, 8), (100_001, 1025, 2)])
@pytest.mark.parametrize("mean", [0.0, 1.0])
def test_weight_gradient_of_many_rows(torch, rows, cols, each, mean):
    """Hundreds of rows a lane: the bound grows with them, also where every term has the same sign."""
    h, dy = normal(torch, 1, rows, cols, dtype="bfloat16") + mean, normal(torch, 2, rows, cols, dtype="bfloat16") + mean
    w, r, add = normal(torch, 3, cols) + 1, torch.empty(rows, device="cuda"), normal(torch, 4, cols)
    L.demo_rms_norm(L.Norm(), h, w, rstd=r)
    work = torch.empty(L.demo_rms_norm_workspace(L.Norm(), rows, cols), dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(h), add.clone()
    L.demo_rms_norm_backward(L.Norm(), dy, h, w, r, dx, dweight=dw, addend=dw, workspace=work)
    check_dw(torch, dw, dy, h, r, add, -(-rows // (each * 512)))
