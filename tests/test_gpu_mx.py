"""The linear layer on 4-bit operands on the GPU against its 64-bit forms.

Tolerances.  u is half a step of the result's type (finfo.eps / 2).
  quantise  scaling by a power of two is exact: codes and exponents are equal.
  values    code times scale is exact, then one rounding to the type.
  product   products of two codes are multiples of 1/4 up to 36, which a matrix
            instruction keeps; it adds 16 groups of 8 neighbours and the sum so
            far, each kept down to 2^-23 of the largest one, so 128 of the sum
            are off by at most 17 2^-23 S, S = sum |a b|.  Sums of waves and of
            splits are 64 more: (17 ceil(k/128) + 64) 2^-23 S + 2^-23 |result| +
            u |result|, plus half the type's smallest step.  Sums in fp32 without
            matrix instructions are within that: one rounding a product at most.
"""
import threading

import linear_forms as F
import numpy as np
import pytest
import train_forms as T

from communication_compressed_optimizer_elt_amd import binding as L

pytestmark = pytest.mark.gpu
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


def operand(torch, rows, cols):
    return torch.full((L.demo_mx_layout(rows, cols)["total_bytes"],), 0xA5, dtype=torch.uint8, device="cuda")


def check_operand(buf, x, tile):
    codes, e, clean = T.mx_unpack(buf.cpu().numpy(), *x.shape)
    want, we = T.mx_quantize(x, tile)
    assert np.array_equal(e, we)
    assert np.array_equal(codes, want)
    assert clean


# ----------------------------------------------------------------- quantise --

@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (32, 1), (1, 300), (3, 7), (31, 33), (128, 128), (130, 257), (300, 1000),
                                       (5, 4096), (1025, 640), (64, 517), (257, 512)])
@pytest.mark.parametrize("tile", [0, 1])
@pytest.mark.parametrize("dtype", DT)
def test_quantize(torch, rows, cols, tile, dtype):
    x = normal(torch, rows + cols, rows, cols, dtype=dtype)
    x *= torch.exp2(torch.arange(cols, device="cuda") % 7 - 3.0).to(x.dtype)
    q, qt = operand(torch, rows, cols), operand(torch, cols, rows)
    L.demo_mx_quantize(L.Mx(tile=tile), x, q, qt)
    check_operand(q, host(x), tile)
    check_operand(qt, host(x).T, tile)
    one, other = operand(torch, rows, cols), operand(torch, cols, rows)
    L.demo_mx_quantize(L.Mx(tile=tile), x, operand=one)
    L.demo_mx_quantize(L.Mx(tile=tile), x, operand_t=other)
    check_operand(one, host(x), tile)
    check_operand(other, host(x).T, tile)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("cols,pitch,at", [(200, 256, 0), (200, 301, 1), (256, 384, 128), (33, 40, 3)])
def test_quantize_slices(torch, dtype, cols, pitch, at):
    x = normal(torch, 7, 140, pitch, dtype=dtype)[:, at: at + cols]
    q, qt = operand(torch, 140, cols), operand(torch, cols, 140)
    L.demo_mx_quantize(L.Mx(), x, q, qt)
    check_operand(q, host(x), 0)
    check_operand(qt, host(x).T, 0)


def test_quantize_every_rounding(torch):
    """Every middle between two codes, both neighbours of it, both signs, at
    scales over the whole range; blocks whose maximum lies next to a border."""
    v = np.concatenate([[m, np.nextafter(np.float32(m), np.float32(9)), np.nextafter(np.float32(m), np.float32(-9))]
                        for m in (0.25, 0.5, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.0)])
    v = np.concatenate([v, -v]).astype(np.float32)
    rows = []
    for e in (-127, -126, -120, -100, -30, -3, 0, 1, 40, 100, 124, 125):
        for top in (6.0, np.nextafter(np.float32(6), np.float32(0)), np.nextafter(np.float32(6), np.float32(9)), 4.0, 3.5):
            row = np.ldexp(np.concatenate([v[:31], [top], v[23:], [top]]).astype(np.float64), e)
            rows.append(np.resize(row, 64))
    x = torch.tensor(np.array(rows)).float()
    x = torch.cat([x, torch.zeros(2, 64), -torch.zeros(1, 64), torch.full((1, 64), 1e-45)]).cuda()
    q, qt = operand(torch, *x.shape), operand(torch, 64, x.shape[0])
    L.demo_mx_quantize(L.Mx(), x, q, qt)
    check_operand(q, host(x), 0)
    check_operand(qt, host(x).T, 0)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_quantize_every_16_bit_value(torch, dtype):
    """All finite values of a 16-bit type, each in a block with a larger one."""
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(getattr(torch, dtype)).float()
    x = x[torch.isfinite(x)]
    x = x[x.abs().argsort()][: x.numel() // 32 * 32].view(-1, 32).to(getattr(torch, dtype)).cuda()
    q = operand(torch, *x.shape)
    L.demo_mx_quantize(L.Mx(), x, q)
    check_operand(q, host(x), 0)


@pytest.mark.parametrize("tile", [0, 1])
@pytest.mark.parametrize("dtype", DT)
def test_quantize_infinities_and_nan(torch, tile, dtype):
    x = normal(torch, 9, 200, 300, dtype=dtype)
    x[3, 5], x[3, 200], x[150, 20], x[199, 299] = float("inf"), float("nan"), -float("inf"), float("nan")
    q, qt = operand(torch, 200, 300), operand(torch, 300, 200)
    L.demo_mx_quantize(L.Mx(tile=tile), x, q, qt)
    check_operand(q, host(x), tile)
    check_operand(qt, host(x).T, tile)
    y = torch.empty(200, 300, device="cuda")
    L.demo_mx_dequantize(q, y)
    codes, e = T.mx_quantize(host(x), tile)
    assert np.array_equal(host(y), T.mx_value(codes, e), equal_nan=True)
    assert torch.isnan(y[3, 5]) and not torch.isnan(y[100, 290])


@pytest.mark.parametrize("p", [0.1, 0.5, 1.0])
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,cols", [(130, 264), (65, 77)])
def test_quantize_through_a_dropout(torch, p, dtype, rows, cols):
    x = normal(torch, 5, rows, cols, dtype=dtype)
    kw = dict(p=p, seed=77, step=5, site=3, chunk_offset=11)
    q, qt = operand(torch, rows, cols), operand(torch, cols, rows)
    for tile in (0, 1):
        L.demo_mx_quantize(L.Mx(tile=tile), x, q, qt, dropout=L.Dropout(**kw))
        want = T.dropped(host(x), **kw)
        check_operand(q, want, tile)
        check_operand(qt, want.T, tile)


def test_squares_quantise_alike_both_ways(torch):
    x = normal(torch, 5, 160, 224)
    q, qt = operand(torch, 160, 224), operand(torch, 224, 160)
    a, b = torch.empty(160, 224, device="cuda"), torch.empty(224, 160, device="cuda")
    L.demo_mx_quantize(L.Mx(tile=1), x, q, qt)
    L.demo_mx_dequantize(q, a)
    L.demo_mx_dequantize(qt, b)
    assert torch.equal(a, b.t())


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,cols,pitch,at", [(1, 1, 1, 0), (3, 40, 40, 0), (130, 257, 300, 1), (64, 512, 640, 64)])
def test_values(torch, dtype, rows, cols, pitch, at):
    x = normal(torch, 5, rows, cols) * torch.exp2(torch.arange(cols, device="cuda") % 40 - 20.0)
    q = operand(torch, rows, cols)
    L.demo_mx_quantize(L.Mx(), x, q)
    wide = torch.full((rows, pitch), 7.0, dtype=getattr(torch, dtype), device="cuda")
    L.demo_mx_dequantize(q, wide[:, at: at + cols])
    want = torch.full((rows, pitch), 7.0, dtype=torch.float64)
    want[:, at: at + cols] = torch.from_numpy(T.mx_value(*T.mx_quantize(host(x), 0)))
    assert torch.equal(wide.cpu(), want.to(getattr(torch, dtype)))


def test_values_at_the_ends_of_the_range(torch):
    e = np.array([[-127, -126, 0, 126, 127, 128]])
    codes = np.resize(np.concatenate([T.GRID, -T.GRID[1:]]), (1, 192))
    buf = torch.from_numpy(T.mx_pack(codes, e)).cuda()
    y = torch.empty(1, 192, device="cuda")
    L.demo_mx_dequantize(buf, y)
    with np.errstate(over="ignore"):
        assert np.array_equal(host(y), T.mx_value(codes, e).astype(np.float32).astype(np.float64), equal_nan=True)


# ------------------------------------------------------------------ product --

def packed(torch, seed, rows, cols, spread=6):
    """(operand, its values) of random codes and exponents."""
    g = np.random.default_rng(seed)
    codes = g.choice(np.concatenate([T.GRID, -T.GRID]), (rows, cols))
    e = g.integers(-spread, spread + 1, (rows, -(-cols // 32)))
    return torch.from_numpy(T.mx_pack(codes, e)).cuda(), T.mx_value(codes, e)


def check_product(torch, c, a, b, addend=None, mask=None, scale=1.0):
    want, s = a @ b.T, np.abs(a) @ np.abs(b).T
    k = a.shape[1]
    f = torch.finfo(c.dtype)
    if mask is not None:
        want, s = want * scale * mask, s * scale * mask
    err = (17 * -(-k // 128) + 64) * 2.0**-23 * s + 2.0**-23 * np.abs(want)
    if addend is not None:
        want = want + host(addend)
        err = err + 2.0**-23 * (np.abs(host(addend)) + np.abs(want))
    bound = err + f.eps / 2 * (np.abs(want) + err) + f.tiny * f.eps / 2
    got = host(c)
    over = np.abs(want) + err >= f.max
    assert (np.isinf(got) | (np.abs(got - want) <= bound))[over].all()
    assert (np.abs(got - want) <= bound)[~over].all()


def workspace(torch, m, n, k, dtype="float32"):
    need = L.demo_mx_workspace(L.Mx(), m, n, k, getattr(L, {"float32": "DTYPE_F32", "float16": "DTYPE_F16", "bfloat16": "DTYPE_BF16"}[dtype]))
    return torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")


SIZES = [(1, 1, 1), (1, 17, 300), (1, 2048, 1024), (2, 33, 257), (3, 64, 31), (4, 100, 5000), (9, 70, 640), (16, 64, 256), (17, 65, 255),
         (64, 64, 512), (129, 127, 1000), (300, 260, 2561), (64, 64, 16384), (40, 200, 9000), (256, 256, 512), (257, 300, 256),
         (600, 520, 1300), (2304, 768, 769), (1024, 2048, 384), (4100, 2060, 520), (2048, 2048, 12288)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", DT)
def test_product(torch, m, n, k, dtype):
    (qa, a), (qb, b) = packed(torch, m + n, m, k), packed(torch, n + k, n, k)
    d = getattr(torch, dtype)
    c = torch.full((m, n), 9.0, dtype=d, device="cuda")
    ws = workspace(torch, m, n, k, dtype)
    L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, c, workspace=ws)
    check_product(torch, c, a, b)
    again = torch.empty_like(c)
    L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, again, workspace=ws)
    assert torch.equal(c, again)
    add = normal(torch, 3, m, n, std=10.0, dtype=dtype)
    acc, other = add.clone(), torch.empty_like(add)
    L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, acc, addend=acc, workspace=ws)
    L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, other, addend=add, workspace=ws)
    assert torch.equal(acc, other)
    check_product(torch, acc, a, b, add)


@pytest.mark.parametrize("k", [100, 257, 520, 1024, 1100, 1500, 2000])
@pytest.mark.parametrize("m,n", [(4100, 2060), (2100, 4104)])
def test_large_product(torch, m, n, k):
    """Tiles of 256 with every number of steps up to 8, moved back inside at both ends."""
    (qa, a), (qb, b) = packed(torch, k, m, k), packed(torch, n, n, k)
    c = torch.full((m, n), 9.0, dtype=torch.bfloat16, device="cuda")
    add = normal(torch, 3, m, n, std=10.0)
    acc = add.clone()
    L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, c)
    L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, acc, addend=acc)
    check_product(torch, c, a, b)
    check_product(torch, acc, a, b, add)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("k", [1024, 1500, 2048, 2300])
def test_several_tiles_a_workgroup(torch, k, dtype):
    """561 tiles of 256: up to three one after another, the last ones moved back inside."""
    m, n = 8200, 4104
    (qa, a), (qb, b) = packed(torch, k, m, k), packed(torch, n, n, k)
    c = torch.full((m + 1, n), 9.0, dtype=getattr(torch, dtype), device="cuda")
    L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, c[:m])
    assert (c[m] == 9.0).all()
    a, b = torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda()
    want, s = a @ b.t(), a.abs() @ b.abs().t()
    f = torch.finfo(c.dtype)
    err = (17 * -(-k // 128) + 64) * 2.0**-23 * s + 2.0**-23 * want.abs()
    bound = err + f.eps / 2 * (want.abs() + err) + f.tiny * f.eps / 2
    over = (want.abs() + err >= f.max) & c[:m].isinf() & (c[:m] * want > 0)  # as in check_product
    assert (over | ((c[:m].double() - want).abs() <= bound)).all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("m,n,k", [(1, 70, 300), (2, 70, 300), (12, 70, 300), (140, 133, 300), (300, 270, 600), (64, 64, 16384)])
def test_product_slices(torch, dtype, m, n, k):
    """Results and addends that are slices of wider matrices, aligned and not."""
    (qa, a), (qb, b) = packed(torch, 1, m, k), packed(torch, 2, n, k)
    ws = workspace(torch, m, n, k, dtype)
    for pitch, at in ((n + 11, 3), (-(-n // 8) * 8 + 64, 8)):
        wide, add = (normal(torch, s, m, pitch, dtype=dtype) for s in (4, 5))
        before = wide.clone()
        L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, wide[:, at: at + n], addend=add[:, at: at + n], workspace=ws)
        check_product(torch, wide[:, at: at + n], a, b, add[:, at: at + n])
        wide[:, at: at + n] = 0
        before[:, at: at + n] = 0
        assert torch.equal(wide, before)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("m,n,k", [(1, 72, 300), (2, 70, 300), (12, 72, 300), (140, 136, 300), (140, 133, 300), (512, 512, 300), (64, 64, 16384)])
def test_product_through_a_dropout(torch, dtype, m, n, k):
    (qa, a), (qb, b) = packed(torch, 1, m, k), packed(torch, 2, n, k)
    kw = dict(p=0.25, seed=9, step=4, site=2, chunk_offset=3)
    add = normal(torch, 5, m, n, dtype=dtype)
    c = torch.empty_like(add)
    L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, c, addend=add, dropout=L.Dropout(**kw), workspace=workspace(torch, m, n, k, dtype))
    check_product(torch, c, a, b, add, F.keep(m * n, **kw).reshape(m, n), F.scale(0.25))


@pytest.mark.parametrize("m,n", [(1, 40), (2, 40), (7, 40), (70, 80), (300, 300), (512, 2100)])
def test_product_of_nan_blocks(torch, m, n):
    """A block of scale byte 255 makes its row, or its column, NaN and leaves the others."""
    k = 700
    g = np.random.default_rng(3)
    ca, cb = (g.choice(T.GRID, (r, k)) for r in (m, n))
    ea, eb = (g.integers(-3, 4, (r, 22)) for r in (m, n))
    eb[5, 21] = eb[11, 0] = 128
    bad_row = m - 1
    if m > 1:
        ea[bad_row, 7] = 128
    c = torch.empty(m, n, device="cuda")
    L.demo_mx_matmul(L.Mx(), m, n, k, torch.from_numpy(T.mx_pack(ca, ea)).cuda(), torch.from_numpy(T.mx_pack(cb, eb)).cuda(), c,
                     workspace=workspace(torch, m, n, k))
    want = T.mx_value(ca, ea) @ T.mx_value(cb, eb).T
    assert np.isnan(want[:, 5]).all() and np.isnan(want).sum() == 2 * m + (n - 2 if m > 1 else 0)
    assert np.array_equal(np.isnan(host(c)), np.isnan(want))


@pytest.mark.parametrize("m,n", [(1, 40), (2, 40), (7, 40), (70, 80), (300, 300)])
def test_product_scales_far_from_one(torch, m, n):
    """Scales at the ends: products of large and small blocks that meet in the middle, and zero rows."""
    k = 512
    g = np.random.default_rng(4)
    ca, cb = (g.choice(np.concatenate([T.GRID, -T.GRID]), (r, k)) for r in (m, n))
    ea, eb = np.full((m, 16), -120), np.full((n, 16), 118)
    ca[0, :256] = 0
    cb[n // 2] = 0
    c = torch.empty(m, n, device="cuda")
    L.demo_mx_matmul(L.Mx(), m, n, k, torch.from_numpy(T.mx_pack(ca, ea)).cuda(), torch.from_numpy(T.mx_pack(cb, eb)).cuda(), c,
                     workspace=workspace(torch, m, n, k))
    check_product(torch, c, T.mx_value(ca, ea), T.mx_value(cb, eb))


def test_small_integers_are_exact(torch):
    """Sums of integers below 2^24 are exact in any order; spread scales keep them integers."""
    m, n, k = 130, 140, 4096
    g = np.random.default_rng(6)
    for rows in (1, 2, 8, m):
        ca, cb = g.choice([0, 1, 2, 3, 4, 6, -1, -2, -3], (rows, k)), g.choice([0, 1, 2, 3, 4, 6, -1, -2, -3], (n, k))
        ea, eb = g.integers(0, 3, (rows, k // 32)), g.integers(0, 3, (n, k // 32))
        c = torch.empty(rows, n, device="cuda")
        L.demo_mx_matmul(L.Mx(), rows, n, k, torch.from_numpy(T.mx_pack(ca.astype(float), ea)).cuda(),
                         torch.from_numpy(T.mx_pack(cb.astype(float), eb)).cuda(), c, workspace=workspace(torch, rows, n, k))
        assert np.array_equal(host(c), T.mx_value(ca.astype(float), ea) @ T.mx_value(cb.astype(float), eb).T)


# -------------------------------------------------------------------- layer --

def test_layer_forward_and_backward(torch):
    """Y = residual + drop(X W^T), dX and dW through the operators, each against 64 bits on the values its operands hold."""
    m, n, k = 390, 264, 520
    x, w = normal(torch, 1, m, k, dtype="bfloat16"), normal(torch, 2, n, k, std=0.05)
    res, dy = normal(torch, 3, m, n, dtype="bfloat16"), normal(torch, 4, m, n, std=0.1, dtype="bfloat16")
    kw = dict(p=0.1, seed=5, step=6, site=7)
    mask = F.keep(m * n, **kw).reshape(m, n)
    wq, wt, xq, xt = operand(torch, n, k), operand(torch, k, n), operand(torch, m, k), operand(torch, k, m)
    gq, gt = operand(torch, m, n), operand(torch, n, m)
    ws = torch.empty(L.BLOCK_MAX_WORKSPACE, dtype=torch.uint8, device="cuda")
    y, dx, grad = torch.empty_like(res), torch.empty_like(x), normal(torch, 8, n, k)
    before = grad.clone()
    L.demo_mx_quantize(L.Mx(tile=1), w, wq, wt)
    L.demo_mx_quantize(L.Mx(), x, xq, xt)
    L.demo_mx_matmul(L.Mx(), m, n, k, xq, wq, y, addend=res, dropout=L.Dropout(**kw), workspace=ws)
    L.demo_mx_quantize(L.Mx(), dy, gq, gt, dropout=L.Dropout(**kw))
    L.demo_mx_matmul(L.Mx(), m, k, n, gq, wt, dx, workspace=ws)
    L.demo_mx_matmul(L.Mx(), n, k, m, gt, xt, grad, addend=grad, workspace=ws)
    v = lambda t, tile=0: T.mx_value(*T.mx_quantize(t, tile))  # noqa: E731
    dropped = T.dropped(host(dy), **kw)
    check_product(torch, y, v(host(x)), v(host(w), 1), res, mask, F.scale(0.1))
    check_product(torch, dx, v(dropped), v(host(w).T, 1))
    check_product(torch, grad, v(dropped.T), v(host(x).T), before)


def test_two_threads_two_streams(torch):
    m, n, k = 64, 64, 16384  # split: each stream has a workspace of its own
    (qa, a), (qb, b) = packed(torch, 1, m, k), packed(torch, 2, n, k)
    out, errors = [torch.empty(m, n, device="cuda") for _ in range(2)], []
    torch.cuda.synchronize()

    def run(i):
        try:
            s, ws = torch.cuda.Stream(), workspace(torch, m, n, k)
            for _ in range(20):
                L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, out[i], workspace=ws, stream=s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    check_product(torch, out[0], a, b)
    assert torch.equal(out[0], out[1])
