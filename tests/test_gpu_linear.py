"""The low-precision linear layer on the GPU against its plain 64-bit forms.

Tolerances.  u is half a step of the result's type (finfo.eps / 2), 2^-24 half
a step of fp32.
  dropout   one fp32 product, one fp32 sum, one rounding to the type:
            2^-24 (|x s| + |y|) + u |y|, plus half the type's smallest step.
  quantise  scaling by a power of two is exact: codes and exponents are equal.
  product   products of codes are exact; a sum takes at most 64 additions in an
            instruction and two more for each block of 128, each off by at most
            a step of fp32 (2^-23, a truncating adder included) of a partial sum
            that is at most S = sum |a b|; joining splits adds at most 64 more:
            (128 + 2 blocks) 2^-23 S + 2^-23 |result| + u |result|.
            16-bit results come from the 8-bit matrix instructions, whose own
            arithmetic is: products are summed in groups of 8 neighbours along
            the sum, each kept down to 2^-13 of the group's largest one, and an
            instruction adds its 16 groups and the sum so far, each kept down
            to 2^-23 of the largest.  So a group's 8 products are off by less
            than 8 * 2^-13 max|a b| <= 2^-10 max|a| max|b| together, and a
            block's 17 addends by 17 * 2^-23 S:
            2^-10 sum over groups of max|a| max|b| + (17 blocks + 64) 2^-23 S
            + 2^-23 |result| + u |result|.
"""
import threading

import linear_forms as F
import numpy as np
import pytest

from communication_compressed_optimizer_elt_amd import binding as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    L.lib()
    return torch


DT = {"f32": ("float32", L.DTYPE_F32), "f16": ("float16", L.DTYPE_F16), "bf16": ("bfloat16", L.DTYPE_BF16)}


def dt(torch, name):
    return getattr(torch, DT[name][0])


def host(t):
    return t.detach().double().cpu().numpy()


def half_step(torch, dtype):
    f = torch.finfo(dtype)
    return f.eps / 2, f.tiny * f.eps / 2  # relative, and absolute below the normals


def normal(torch, seed, *shape, std=1.0, dtype=None):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype or torch.float32).cuda()


def check_dropped(torch, y, x, residual, mask, p):
    xs = host(x) * F.scale(p) * mask.reshape(x.shape)
    want = xs + (host(residual) if residual is not None else 0)
    u, low = half_step(torch, y.dtype)
    err = np.abs(host(y) - want)
    bound = 2.0**-24 * (np.abs(xs) + np.abs(want)) + u * np.abs(want) * (1 + 2.0**-20) + low
    assert (err <= bound).all(), (err - bound).max()


# ------------------------------------------------------------------ dropout --

@pytest.mark.parametrize("n", [1, 7, 8, 9, 2047, 2048, 2049, 100_003])
@pytest.mark.parametrize("dtype", sorted(DT))
def test_dropout(torch, n, dtype):
    d = dt(torch, dtype)
    x, r = normal(torch, n, n, dtype=d), normal(torch, n + 1, n, std=3.0, dtype=d)
    cfg = dict(p=0.1, seed=0x1234567_89ABCDEF, step=(5 << 32) + 77, site=n % 9, chunk_offset=12345)
    mask = F.keep(n, **cfg)
    y = torch.full_like(x, 9.0)
    L.demo_dropout(L.Dropout(**cfg), x, y)
    check_dropped(torch, y, x, None, mask, 0.1)
    L.demo_dropout(L.Dropout(**cfg), x, y, residual=r)
    check_dropped(torch, y, x, r, mask, 0.1)
    dx = torch.empty_like(x)
    L.demo_dropout_backward(L.Dropout(**cfg), x, dx)
    check_dropped(torch, dx, x, None, mask, 0.1)
    if n > 10_000:  # the share kept: 5 standard deviations
        assert abs(mask.mean() - 0.9) < 5 * (0.09 / n) ** 0.5


@pytest.mark.parametrize("p", [0.0, 1e-6, 2.0**-16, 0.5, 0.999, 1.0 - 2.0**-16, 1.0])
def test_dropout_probabilities(torch, p):
    n = 4099
    x = normal(torch, 3, n)
    y = torch.empty_like(x)
    L.demo_dropout(L.Dropout(p=p, seed=8), x, y)
    check_dropped(torch, y, x, None, F.keep(n, p, seed=8), p)
    if p == 0.0:
        assert torch.equal(x, y)
    if p == 1.0:
        assert not y.any()


def test_dropout_in_place_and_shards(torch):
    n = 32 * 700 + 5
    x, r = normal(torch, 4, n), normal(torch, 5, n)
    d = L.Dropout(p=0.3, seed=11, step=2)
    y = torch.empty_like(x)
    L.demo_dropout(d, x, y, residual=r)
    a = x.clone()
    L.demo_dropout(d, a, a, residual=r)
    b = r.clone()
    L.demo_dropout(d, x, b, residual=b)
    assert torch.equal(a, y) and torch.equal(b, y)
    part = torch.empty_like(x)  # two shards draw what the whole tensor draws
    cut = 32 * 301
    L.demo_dropout(L.Dropout(p=0.3, seed=11, step=2), x[:cut], part[:cut], residual=r[:cut])
    tail = torch.empty(n - cut, device="cuda")
    L.demo_dropout(L.Dropout(p=0.3, seed=11, step=2, chunk_offset=301), x[cut:].clone(), tail, residual=r[cut:].clone())
    assert torch.equal(torch.cat([part[:cut], tail]), y)


def test_dropout_leaves_nothing_of_what_it_drops(torch):
    n = 4096
    mask = torch.from_numpy(F.keep(n, 0.5, seed=3)).cuda()
    x = torch.where(mask, 1.0, float("nan"))
    x[5:40] = torch.where(mask[5:40], 1.0, float("inf"))
    y = torch.empty_like(x)
    L.demo_dropout(L.Dropout(p=0.5, seed=3), x, y)
    assert torch.equal(y, torch.where(mask, 2.0, 0.0))
    x = torch.where(mask, float("nan"), 1.0)
    L.demo_dropout_backward(L.Dropout(p=0.5, seed=3), x, y)
    assert torch.equal(torch.isnan(y), mask)


def test_dropout_streams_of_numbers_differ(torch):
    n = 32768
    x = torch.ones(n, device="cuda")
    seen = []
    for kw in (dict(), dict(seed=1), dict(seed=1 << 32), dict(step=1), dict(site=1), dict(chunk_offset=1)):
        y = torch.empty_like(x)
        L.demo_dropout(L.Dropout(p=0.5, **kw), x, y)
        seen.append(y.bool())
    for i in range(len(seen)):
        for j in range(i):
            agree = float((seen[i] == seen[j]).double().mean())  # 8 standard deviations of a fair coin
            assert abs(agree - 0.5) < 8 * 0.5 / n**0.5, (i, j)


def test_dropout_beyond_2_pow_32_elements(torch):
    """The tail behind element 2^32 of one call draws what a call of the tail alone draws."""
    n = (1 << 32) + 4099
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros_like(x)
    L.demo_dropout(L.Dropout(p=0.25, seed=9), x, y)
    at = (1 << 32) - 64
    tail = host(y[at:])
    mask = F.keep(n - at, 0.25, seed=9, chunk_offset=at // 32)
    assert np.array_equal(tail != 0, mask)


def test_dropout_gradient_by_differences(torch):
    """The operator is linear in x and residual: with powers of two the central
    differences of sum(dy * y) are the gradients exactly."""
    n = 512
    d = L.Dropout(p=0.5, seed=21)
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-8, 9, (n,), generator=g).float().cuda()
    dy = torch.randint(-8, 9, (n,), generator=g).float().cuda()

    def loss(x, r):
        y = torch.empty_like(x)
        L.demo_dropout(d, x, y, residual=r)
        return float((dy * y).sum())

    dx = torch.empty_like(x)
    L.demo_dropout_backward(d, dy, dx)
    for i in (0, 1, 7, 8, 100, 511):
        e = torch.zeros_like(x)
        e[i] = 1.0
        assert (loss(x + e, x) - loss(x - e, x)) / 2 == float(dx[i])
        assert (loss(x, x + e) - loss(x, x - e)) / 2 == float(dy[i])


# ----------------------------------------------------------------- quantise --

def check_operand(torch, buf, x, fmt, tile):
    codes, e, clean = F.unpack(buf.cpu().numpy(), *x.shape, fmt)
    want, we = F.quantize(x, fmt, tile)
    assert np.array_equal(e, we)
    assert np.array_equal(codes, want, equal_nan=True)
    assert clean


def operand(torch, rows, cols):
    return torch.full((L.demo_block_layout(rows, cols)["total_bytes"],), 0xA5, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (128, 1), (3, 7), (127, 129), (128, 128), (130, 257), (300, 1000),
                                       (5, 4096), (1025, 640), (64, 517)])
@pytest.mark.parametrize("fmt", [L.FMT_E4M3, L.FMT_E5M2])
@pytest.mark.parametrize("tile", [0, 1])
@pytest.mark.parametrize("dtype", sorted(DT))
def test_quantize(torch, rows, cols, fmt, tile, dtype):
    x = normal(torch, rows + cols, rows, cols, dtype=dt(torch, dtype))
    x *= torch.exp2(torch.arange(cols, device="cuda") % 7 - 3.0).to(x.dtype)
    q, qt = operand(torch, rows, cols), operand(torch, cols, rows)
    L.demo_block_quantize(L.Block(fmt=fmt, tile=tile), x, q, qt)
    check_operand(torch, q, host(x), fmt, tile)
    check_operand(torch, qt, host(x).T, fmt, tile)
    one, other = operand(torch, rows, cols), operand(torch, cols, rows)
    L.demo_block_quantize(L.Block(fmt=fmt, tile=tile), x, operand=one)
    L.demo_block_quantize(L.Block(fmt=fmt, tile=tile), x, operand_t=other)
    for a, b, (r, c) in ((q, one, (rows, cols)), (qt, other, (cols, rows))):
        for u, v in zip(F.unpack(a.cpu().numpy(), r, c, fmt), F.unpack(b.cpu().numpy(), r, c, fmt)):
            assert np.array_equal(u, v, equal_nan=True) if u is not True else v


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("cols,pitch,at", [(200, 256, 0), (200, 301, 1), (256, 384, 128), (33, 40, 3)])
def test_quantize_slices(torch, dtype, cols, pitch, at):
    """A column slice of a wider matrix, aligned and not."""
    wide = normal(torch, 7, 140, pitch, dtype=dt(torch, dtype))
    x = wide[:, at: at + cols]
    q, qt = operand(torch, 140, cols), operand(torch, cols, 140)
    L.demo_block_quantize(L.Block(), x, q, qt)
    check_operand(torch, q, host(x), 0, 0)
    check_operand(torch, qt, host(x).T, 0, 0)


@pytest.mark.parametrize("fmt", [0, 1])
def test_quantize_edges_of_the_range(torch, fmt):
    """Block maxima next to every power of two and next to fmax times one,
    subnormals, zeros of both signs, values that underflow."""
    top = F.FORMATS[fmt][0]
    rows = []
    for e in (-149, -140, -135, -127, -126, -120, -118, -100, -20, -1, 0, 1, 8, 9, 15, 16, 60, 110, 118, 119):
        for m in (1.0, 1.0 + 2.0**-23, 1.75, 1.75 + 2.0**-23, 2.0 - 2.0**-23):
            x = np.float32(0) + np.ldexp(np.float64(m), e)
            rows.append([x if x <= 3.4e38 else 3.4e38] + [x * 2.0**-j * s for j in range(1, 60) for s in (1, -0.75)])
    x = torch.tensor(np.array(rows), dtype=torch.float64).float()
    x = torch.cat([x, torch.zeros(2, x.shape[1]), -torch.zeros(1, x.shape[1])]).cuda()
    q, qt = operand(torch, *x.shape), operand(torch, x.shape[1], x.shape[0])
    L.demo_block_quantize(L.Block(fmt=fmt), x, q, qt)
    check_operand(torch, q, host(x), fmt, 0)
    check_operand(torch, qt, host(x).T, fmt, 0)
    assert top > 0


@pytest.mark.parametrize("tile", [0, 1])
@pytest.mark.parametrize("fmt", [0, 1])
def test_quantize_infinities_and_nan(torch, fmt, tile):
    x = normal(torch, 9, 200, 300)
    x[3, 5], x[3, 200], x[150, 20], x[199, 299] = float("inf"), float("nan"), -float("inf"), float("nan")
    x[7] = float("nan")
    x[8, :128] = float("inf")
    q, qt = operand(torch, 200, 300), operand(torch, 300, 200)
    L.demo_block_quantize(L.Block(fmt=fmt, tile=tile), x, q, qt)
    check_operand(torch, q, host(x), fmt, tile)
    check_operand(torch, qt, host(x).T, fmt, tile)


@pytest.mark.parametrize("rows,cols", [(130, 256), (129, 131), (3, 5), (256, 250)])
@pytest.mark.parametrize("dtype", sorted(DT))
def test_quantize_with_dropout(torch, rows, cols, dtype):
    x = normal(torch, 10, rows, cols, dtype=dt(torch, dtype))
    x[0, 0] = float("nan")
    kw = dict(p=0.2, seed=77, step=3, site=2, chunk_offset=9)
    q, qt = operand(torch, rows, cols), operand(torch, cols, rows)
    L.demo_block_quantize(L.Block(fmt=1), x, q, qt, dropout=L.Dropout(**kw))
    g = np.float32(host(x)) * np.float32(F.scale(0.2))  # fp32, rounded once
    g = np.where(F.keep(rows * cols, **kw).reshape(rows, cols), g, np.float32(0))
    check_operand(torch, q, g, 1, 0)
    check_operand(torch, qt, g.T, 1, 0)


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0 - 2.0**-16, 1.0])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cols", [200, 203])
def test_quantize_with_dropout_at_the_range_end(torch, cols, dtype, p):
    """Kept values whose product with the scale overflows fp32 are infinite:
    NaN codes, and no part of a block's largest magnitude.  What is dropped
    leaves nothing, NaN and infinities included."""
    rows = 140
    x = normal(torch, 14, rows, cols, dtype=dt(torch, dtype))
    top = torch.finfo(x.dtype).max
    x[1::9, ::5] = top
    x[2::9, ::7] = -top * 0.93
    x[3::9, 1::4] = top / 1.99
    x[4::9, 2::11] = float("inf")
    x[5::9, 3::6] = float("nan")
    x[6::9] *= torch.finfo(x.dtype).tiny
    kw = dict(p=p, seed=5, step=1, site=3)
    for tile in (0, 1):
        q, qt = operand(torch, rows, cols), operand(torch, cols, rows)
        L.demo_block_quantize(L.Block(fmt=1, tile=tile), x, q, qt, dropout=L.Dropout(**kw))
        with np.errstate(over="ignore", invalid="ignore"):
            g = np.float32(host(x)) * np.float32(F.scale(p))
        g = np.where(F.keep(rows * cols, **kw).reshape(rows, cols), g, np.float32(0))
        check_operand(torch, q, g, 1, tile)
        check_operand(torch, qt, g.T, 1, tile)


def test_quantize_beyond_2_pow_32_bytes(torch):
    """The last rows of a source and an operand of more than 2^32 elements."""
    rows, cols = (1 << 21) + 130, 2048
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-300:] = normal(torch, 12, 300, cols, dtype=torch.bfloat16)
    q = operand(torch, rows, cols)
    L.demo_block_quantize(L.Block(), x, q)
    lay = L.demo_block_layout(rows, cols)
    codes = q[: rows * lay["pitch"]].view(rows, -1)[-300:].cpu().numpy()
    e = q[lay["scale_off"]: lay["scale_off"] + rows * lay["scale_pitch"]].view(rows, -1)[-300:, :16].cpu().numpy()
    want, we = F.quantize(host(x[-300:]), 0, 0)
    assert np.array_equal(F.decode_codes(codes, 0), want) and np.array_equal(e.astype(np.int64) - 127, we)
    # and the product of those rows with a small operand
    b = normal(torch, 13, 70, cols)
    qb = operand(torch, 70, cols)
    L.demo_block_quantize(L.Block(), b, qb)
    c = torch.full((rows, 70), 5.0, device="cuda")
    L.demo_block_matmul(L.Product(), rows, 70, cols, q, qb, c, workspace=workspace(torch, rows, 70, cols))
    wb = F.value(*F.quantize(host(b), 0, 0))
    check_product(torch, c[-300:], F.value(want, we), wb)
    assert not c[:-300].any()


# ------------------------------------------------------------------ product --

def workspace(torch, m, n, k):
    need = max(L.demo_block_workspace(L.Product(), m, n, k, d) for d in (L.DTYPE_F32, L.DTYPE_BF16))
    return torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None


def check_product(torch, c, a, b, addend=None, mask=None, p=0.0):
    """c against a b^T (values in 64 bits), within the stated tolerance."""
    a, b = (torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in (a, b))
    keep = 1.0 if mask is None else torch.from_numpy(np.ascontiguousarray(mask)).cuda() * F.scale(p)
    want, s = a @ b.t() * keep, a.abs() @ b.abs().t() * keep
    total = want if addend is None else want + addend.cuda().double()
    u, low = half_step(torch, c.dtype)
    blocks = -(-a.shape[1] // 128)
    if c.dtype == torch.float32:
        sums = (128 + 2 * blocks) * 2.0**-23 * s
    else:
        ga, gb = (torch.nn.functional.pad(v.abs(), (0, -v.shape[1] % 8)).unflatten(1, (-1, 8)).amax(2) for v in (a, b))
        sums = 2.0**-10 * (ga @ gb.t()) * keep + (17 * blocks + 64) * 2.0**-23 * s
    bound = sums + 2.0**-23 * (want.abs() + total.abs()) + u * total.abs() * (1 + 2.0**-6) + low
    # from half a step above the type's largest value on, rounding gives infinity
    got, top = c.cuda().double(), torch.finfo(c.dtype).max * (1 + u / 2)
    over = torch.isinf(got)
    assert (total.abs()[over] + bound[over] >= top).all() and (got.sign() == total.sign())[over].all()
    err = torch.where(over, total, got).sub(total).abs()
    assert (err <= bound).all(), (float((err - bound).max()), float(err.max()))


def operands(torch, m, n, k, fa=0, fb=0, seed=0, spread=4):
    """Random code values with exponents that vary by row and block."""
    rng = np.random.default_rng(seed + m * 7 + n * 5 + k)
    out = []
    for rows, fmt in ((m, fa), (n, fb)):
        kb = -(-k // 128)
        v = F.round_to(rng.standard_normal((rows, k)) * 3, fmt)
        e = rng.integers(-spread, spread + 1, (rows, kb))
        out += [torch.from_numpy(F.pack(v, e, fmt)).cuda(), F.value(v, e)]
    return out


SHAPES = [(1, 1, 1), (1, 2048, 8192), (2, 100, 129), (3, 5, 7), (16, 64, 640), (17, 33, 129), (32, 96, 2048), (33, 768, 256),
          (64, 130, 1000), (128, 128, 128), (130, 257, 640), (128, 256, 4096), (300, 515, 513), (1000, 77, 300), (2561, 768, 768),
          (768, 768, 2561), (512, 512, 8192), (515, 1027, 1500), (1, 7, 300), (257, 1, 257), (48, 2050, 520)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("out", sorted(DT))
def test_product(torch, m, n, k, out):
    a, va, b, vb = operands(torch, m, n, k)
    c = torch.full((m, n), float("nan"), dtype=dt(torch, out), device="cuda")
    L.demo_block_matmul(L.Product(), m, n, k, a, b, c, workspace=workspace(torch, m, n, k))
    check_product(torch, c, va, vb)


@pytest.mark.parametrize("m,n,k,out,fa,fb", [
    (2000, 8000, 128, "bf16", 0, 0), (2000, 8000, 300, "f16", 1, 0), (1999, 8000, 385, "bf16", 0, 1), (2048, 8192, 520, "bf16", 1, 1),
    (1801, 7944, 700, "f16", 0, 0), (2000, 8001, 900, "bf16", 0, 0), (1793, 7937, 1100, "f16", 0, 0), (2040, 8184, 2000, "bf16", 0, 0),
    (1000, 5000, 300, "bf16", 0, 0), (1000, 5001, 640, "f16", 1, 1), (1000, 5000, 300, "f32", 1, 0), (2000, 4001, 700, "f32", 0, 0),
    (2000, 8000, 128, "f32", 0, 1), (1999, 8001, 300, "f32", 1, 0), (2040, 8184, 1100, "f32", 1, 1), (1801, 7944, 520, "f32", 0, 0)])
def test_product_large_tiles(torch, m, n, k, out, fa, fb):
    """Sizes of the 256 x 256 tiles, whole and moved back at the ends, sums of 1 to 16 blocks; and of the 128 x 128 tiles."""
    a, va, b, vb = operands(torch, m, n, k, fa, fb, spread=2)
    c = torch.full((m, n), float("nan"), dtype=dt(torch, out), device="cuda")
    cfg = L.Product(fmt_a=fa, fmt_b=fb)
    L.demo_block_matmul(cfg, m, n, k, a, b, c)
    check_product(torch, c, va, vb)
    add = normal(torch, 2, m, n, std=20.0, dtype=c.dtype)
    drop = dict(p=0.25, seed=5, site=2)
    L.demo_block_matmul(cfg, m, n, k, a, b, c, addend=add, dropout=L.Dropout(**drop))
    check_product(torch, c, va, vb, add, F.keep(m * n, **drop).reshape(m, n), 0.25)
    L.demo_block_matmul(cfg, m, n, k, a, b, add, addend=add, dropout=L.Dropout(**drop))
    assert torch.equal(add, c)  # in place: no tile adds twice


@pytest.mark.parametrize("fa,fb", [(0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("m,n,k", [(1, 300, 512), (40, 70, 900), (200, 330, 640), (512, 512, 8192), (1030, 770, 400)])
def test_product_formats(torch, m, n, k, fa, fb):
    a, va, b, vb = operands(torch, m, n, k, fa, fb)
    c = torch.empty(m, n, device="cuda")
    L.demo_block_matmul(L.Product(fmt_a=fa, fmt_b=fb), m, n, k, a, b, c, workspace=workspace(torch, m, n, k))
    check_product(torch, c, va, vb)


@pytest.mark.parametrize("m,n,k", [(1, 2048, 1000), (5, 60, 128), (100, 90, 300), (260, 520, 1024), (512, 512, 8192), (1024, 1024, 512)])
def test_product_of_whole_numbers_is_exact(torch, m, n, k):
    rng = np.random.default_rng(m + n + k)
    va, vb = rng.integers(-8, 9, (m, k)).astype(float), rng.integers(-8, 9, (n, k)).astype(float)
    z = lambda rows: np.zeros((rows, -(-k // 128)), np.int64)  # noqa: E731
    a, b = (torch.from_numpy(F.pack(v, z(len(v)), 0)).cuda() for v in (va, vb))
    c = torch.empty(m, n, device="cuda")
    L.demo_block_matmul(L.Product(), m, n, k, a, b, c, workspace=workspace(torch, m, n, k))
    assert np.array_equal(host(c), va @ vb.T)  # every partial sum below 2^24


@pytest.mark.parametrize("out", ["f16", "bf16"])
def test_product_of_small_whole_numbers_is_exact_in_16_bits(torch, out):
    """|sums| below 2^11 (2^8 in bf16), products within 13 places of each other."""
    top, k = (2, 300) if out == "f16" else (1, 250)
    rng = np.random.default_rng(k)
    for m, n in ((1, 100), (20, 50), (50, 30), (300, 260)):
        va, vb = rng.integers(-top, top + 1, (m, k)).astype(float), rng.integers(-top, top + 1, (n, k)).astype(float)
        z = lambda rows: np.zeros((rows, -(-k // 128)), np.int64)  # noqa: E731
        a, b = (torch.from_numpy(F.pack(v, z(len(v)), 0)).cuda() for v in (va, vb))
        c = torch.empty(m, n, dtype=dt(torch, out), device="cuda")
        L.demo_block_matmul(L.Product(), m, n, k, a, b, c, workspace=workspace(torch, m, n, k))
        assert np.array_equal(host(c), va @ vb.T)


@pytest.mark.parametrize("m,n,k", [(1, 2048, 520), (37, 101, 300), (300, 264, 640), (512, 640, 8192), (1100, 1000, 256)])
@pytest.mark.parametrize("out", sorted(DT))
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_product_with_addend_and_dropout(torch, m, n, k, out, p):
    a, va, b, vb = operands(torch, m, n, k, spread=1)
    d = dt(torch, out)
    add = normal(torch, 1, m, n, std=20.0, dtype=d)
    kw = dict(p=p, seed=5, step=6, site=7, chunk_offset=8)
    mask = F.keep(m * n, **kw).reshape(m, n) if p else None
    drop = L.Dropout(**kw) if p else None
    ws = workspace(torch, m, n, k)
    c = torch.empty(m, n, dtype=d, device="cuda")
    L.demo_block_matmul(L.Product(), m, n, k, a, b, c, addend=add, dropout=drop, workspace=ws)
    check_product(torch, c, va, vb, add, mask, p)
    same = add.clone()  # in place
    L.demo_block_matmul(L.Product(), m, n, k, a, b, same, addend=same, dropout=drop, workspace=ws)
    assert torch.equal(same, c)
    # slices of wider matrices: aligned and odd pitches; what lies between the rows stays
    for pitch, at in ((n + 24 - n % 8, 8), (n + 3, 1)):
        wide, wadd = torch.full((m, pitch), 3.0, dtype=d, device="cuda"), torch.zeros(m, pitch, dtype=d, device="cuda")
        wadd[:, at: at + n] = add
        L.demo_block_matmul(L.Product(), m, n, k, a, b, wide[:, at: at + n], addend=wadd[:, at: at + n], dropout=drop, workspace=ws)
        assert torch.equal(wide[:, at: at + n], c)
        assert (wide[:, :at] == 3).all() and (wide[:, at + n:] == 3).all()


@pytest.mark.parametrize("m", [1, 2, 3, 17])
def test_product_of_millions_of_columns(torch, m):
    """More columns than the grids of the kernels for few rows hold."""
    n, k = (1 << 24) + 70, 128
    x, w = normal(torch, 1, m, k), torch.zeros(n, k, dtype=torch.bfloat16, device="cuda")
    at = [0, 77, (1 << 22) - 1, 1 << 22, (1 << 24) + 69]
    w[at] = normal(torch, 2, len(at), k, dtype=torch.bfloat16)
    a, b = operand(torch, m, k), operand(torch, n, k)
    L.demo_block_quantize(L.Block(), x, a)
    L.demo_block_quantize(L.Block(), w, b)
    c = torch.full((m, n), 3.0, device="cuda")
    L.demo_block_matmul(L.Product(), m, n, k, a, b, c, workspace=workspace(torch, m, n, k))
    check_product(torch, c[:, at], F.value(*F.quantize(host(x), 0, 0)), F.value(*F.quantize(host(w[at]), 0, 0)))
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert not c[:, rest].any()


def test_product_range_of_scales(torch):
    """The smallest and largest scale bytes; zero rows; NaN codes reach their row or column only."""
    m, n, k = 40, 48, 256
    rng = np.random.default_rng(0)
    va, vb = F.round_to(rng.standard_normal((m, k)), 0), F.round_to(rng.standard_normal((n, k)), 0)
    ea, eb = np.zeros((m, 2), np.int64), np.zeros((n, 2), np.int64)
    ea[0], eb[0] = 100, -100
    ea[1], eb[1] = -60, 10
    va[2], ea[2] = 0, -127
    eb[3] = -20
    ea[4, 0], ea[4, 1] = 20, -20
    a, b = F.pack(va, ea, 0), F.pack(vb, eb, 0)
    pitch = F.layout(m, k)[0]
    a[7 * pitch + 130] = 0x7F
    b[9 * pitch + 5] = 0xFF
    c = torch.empty(m, n, device="cuda")
    L.demo_block_matmul(L.Product(), m, n, k, torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda(), c,
                        workspace=workspace(torch, m, n, k))
    got = c.cpu()
    want_nan = torch.zeros(m, n, dtype=torch.bool)
    want_nan[7], want_nan[:, 9] = True, True
    assert torch.equal(torch.isnan(got), want_nan)
    rows, cols = [i for i in range(m) if i != 7], [j for j in range(n) if j != 9]
    check_product(torch, got[rows][:, cols], F.value(va, ea)[rows], F.value(vb, eb)[cols])


def test_product_is_the_same_every_time(torch):
    for m, n, k in ((1, 512, 4096), (512, 512, 8192), (300, 200, 1000), (2048, 2048, 1024), (2500, 1100, 256)):
        a, _, b, _ = operands(torch, m, n, k)
        ws = workspace(torch, m, n, k)
        c = [torch.empty(m, n, device="cuda") for _ in range(3)]
        for x in c:
            L.demo_block_matmul(L.Product(), m, n, k, a, b, x, workspace=ws)
        assert torch.equal(c[0], c[1]) and torch.equal(c[0], c[2])


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_product_split_sum_of_large_tiles(torch, out):
    m, n, k = 1800, 1900, 16500
    a, va, b, vb = operands(torch, m, n, k, spread=1)
    c = torch.empty(m, n, dtype=dt(torch, out), device="cuda")
    L.demo_block_matmul(L.Product(), m, n, k, a, b, c, workspace=workspace(torch, m, n, k))
    check_product(torch, c, va, vb)


def test_product_long_sum(torch):
    """2^20 tokens into a small weight gradient."""
    m, n, k = 48, 64, (1 << 20) + 77
    x, y = normal(torch, 1, k, n, dtype=torch.bfloat16), normal(torch, 2, k, m, dtype=torch.bfloat16)
    a, b = operand(torch, m, k), operand(torch, n, k)
    L.demo_block_quantize(L.Block(fmt=1), y, operand_t=a)
    L.demo_block_quantize(L.Block(), x, operand_t=b)
    c = torch.empty(m, n, device="cuda")
    L.demo_block_matmul(L.Product(fmt_a=1), m, n, k, a, b, c, workspace=workspace(torch, m, n, k))
    va, vb = F.value(*F.quantize(host(y).T, 1, 0)), F.value(*F.quantize(host(x).T, 0, 0))
    check_product(torch, c, va, vb)


# ---------------------------------------------------------------- a layer -----

class Layer:
    """Y = residual + dropout(X W^T) and its backward pass, as a training program calls them."""

    def __init__(self, torch, w, drop, tokens, grad):
        self.torch, self.w, self.drop, self.t, self.grad = torch, w, drop, tokens, grad
        n, k = w.shape
        self.n, self.k = n, k
        self.wq, self.wt = operand(torch, n, k), operand(torch, k, n)
        self.xq, self.xt = operand(torch, tokens, k), operand(torch, k, tokens)
        self.gq, self.gt = operand(torch, tokens, n), operand(torch, n, tokens)
        need = max(L.demo_block_workspace(L.Product(), *s, d) for d in (L.DTYPE_F32, L.DTYPE_BF16) for s in ((tokens, n, k), (tokens, k, n), (n, k, tokens)))
        self.ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")

    def take_weight(self):
        L.demo_block_quantize(L.Block(tile=1), self.w, self.wq, self.wt)

    def forward(self, x, residual, y):
        L.demo_block_quantize(L.Block(), x, self.xq, self.xt)
        L.demo_block_matmul(L.Product(), self.t, self.n, self.k, self.xq, self.wq, y, addend=residual, dropout=self.drop,
                            workspace=self.ws)

    def backward(self, dy, dx):
        L.demo_block_quantize(L.Block(fmt=L.FMT_E5M2), dy, self.gq, self.gt, dropout=self.drop)
        cfg = L.Product(fmt_a=L.FMT_E5M2)
        L.demo_block_matmul(cfg, self.t, self.k, self.n, self.gq, self.wt, dx, workspace=self.ws)
        L.demo_block_matmul(cfg, self.n, self.k, self.t, self.gt, self.xt, self.grad, addend=self.grad, workspace=self.ws)


@pytest.mark.parametrize("tokens,n,k", [(1, 96, 256), (197, 160, 96), (333, 250, 515), (512, 256, 1024)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_layer_forward_and_backward(torch, tokens, n, k, dtype):
    d = dt(torch, dtype)
    w, x = normal(torch, 1, n, k, std=0.05), normal(torch, 2, tokens, k, dtype=d)
    res, dy = normal(torch, 3, tokens, n, dtype=d), normal(torch, 4, tokens, n, std=0.1, dtype=d)
    grad0 = normal(torch, 5, n, k)
    kw = dict(p=0.1, seed=31, step=4, site=5)
    layer = Layer(torch, w, L.Dropout(**kw), tokens, grad0.clone())
    y, dx = torch.empty_like(res), torch.empty(tokens, k, dtype=d, device="cuda")
    layer.take_weight()
    layer.forward(x, res, y)
    layer.backward(dy, dx)
    mask = F.keep(tokens * n, **kw).reshape(tokens, n)
    vx, vw = F.value(*F.quantize(host(x), 0, 0)), F.value(*F.quantize(host(w), 0, 1))
    check_product(torch, y, vx, vw, res, mask, 0.1)
    g = np.where(mask, np.float32(host(dy)) * np.float32(F.scale(0.1)), np.float32(0))
    check_product(torch, dx, F.value(*F.quantize(g, 1, 0)), vw.T)
    check_product(torch, layer.grad, F.value(*F.quantize(g.T, 1, 0)), F.value(*F.quantize(host(x).T, 0, 0)), grad0)


def test_layer_gradients_by_differences(torch):
    """Small whole numbers survive quantisation exactly and the layer is
    bilinear: central differences of sum(dy * y) are the gradients exactly."""
    tokens, n, k = 24, 40, 136
    g = torch.Generator().manual_seed(2)
    w = torch.randint(-4, 5, (n, k), generator=g).float().cuda()
    x = torch.randint(-4, 5, (tokens, k), generator=g).float().cuda()
    dy = torch.randint(-3, 4, (tokens, n), generator=g).float().cuda()
    res = torch.zeros(tokens, n, device="cuda")
    drop = L.Dropout(p=0.5, seed=6)

    def loss(w, x):
        layer = Layer(torch, w, drop, tokens, torch.zeros_like(w))
        y = torch.empty_like(res)
        layer.take_weight()
        layer.forward(x, res, y)
        return float((dy * y).double().sum())

    layer = Layer(torch, w, drop, tokens, torch.zeros_like(w))
    y, dx = torch.empty_like(res), torch.empty_like(x)
    layer.take_weight()
    layer.forward(x, res, y)
    layer.backward(dy, dx)
    for i, j in ((0, 0), (3, 127), (39, 128), (20, 135), (11, 64)):
        e = torch.zeros_like(w)
        e[i, j] = 1.0
        assert (loss(w + e, x) - loss(w - e, x)) / 2 == float(layer.grad[i, j])
    for i, j in ((0, 0), (23, 135), (7, 130)):
        e = torch.zeros_like(x)
        e[i, j] = 1.0
        assert (loss(w, x + e) - loss(w, x - e)) / 2 == float(dx[i, j])


def test_training_steps_with_the_optimizer(torch):
    """The layer's weight is a piece of a shard: forward, backward into the
    shard's gradient, demo_encode, demo_decode_apply, and the weight taken
    again - each step's operands are those of the parameters just written."""
    n, k, tokens = 128, 256, 200
    shard = normal(torch, 1, n * k + 64, std=0.05)
    grad, mom = torch.zeros_like(shard), torch.zeros_like(shard)
    cfg = L.Config(scheme=L.SCHEME_DCT, k=4, lr=1e-2)
    pay = torch.zeros(L.demo_payload_layout(cfg, shard.numel())["total_bytes"], dtype=torch.uint8, device="cuda")
    w, gw = shard[: n * k].view(n, k), grad[: n * k].view(n, k)
    drop = L.Dropout(p=0.1, seed=cfg.seed)
    layer = Layer(torch, w, drop, tokens, gw)
    x, dy = normal(torch, 2, tokens, k, dtype=torch.bfloat16), normal(torch, 3, tokens, n, dtype=torch.bfloat16)
    y, dx = torch.empty(tokens, n, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
    res = torch.zeros_like(y)
    for t in range(3):
        before = w.clone()
        grad.zero_()
        cfg.step = drop.step = t
        layer.take_weight()
        layer.forward(x, res, y)
        layer.backward(dy, dx)
        mask = F.keep(tokens * n, 0.1, seed=cfg.seed, step=t).reshape(tokens, n)
        check_product(torch, y, F.value(*F.quantize(host(x), 0, 0)), F.value(*F.quantize(host(before), 0, 1)), res, mask, 0.1)
        g = np.where(mask, np.float32(host(dy)) * np.float32(F.scale(0.1)), np.float32(0))
        check_product(torch, gw, F.value(*F.quantize(g.T, 1, 0)), F.value(*F.quantize(host(x).T, 0, 0)), torch.zeros_like(gw))
        assert not grad[n * k:].any()
        L.demo_encode(cfg, shard.numel(), grad, mom, pay)
        L.demo_decode_apply(cfg, shard.numel(), shard, pay, pay.numel(), 1)
        assert (w != before).any()


# --------------------------------------------- streams, graphs, arguments -----

def test_two_graphs_and_eager_calls_between(torch):
    """Two captured layers with workspaces of their own, replayed in turn with
    eager calls and synchronisations between: every replay as the eager run."""
    made = []
    for i, (tokens, n, k) in enumerate(((512, 512, 2048), (1, 768, 1024))):
        layer = Layer(torch, normal(torch, i, n, k, std=0.05), L.Dropout(p=0.1, seed=i), tokens, torch.zeros(n, k, device="cuda"))
        x, dy = (normal(torch, 10 + i, tokens, c, dtype=torch.bfloat16) for c in (k, n))
        res, y, dx = torch.zeros_like(dy), torch.empty_like(dy), torch.empty_like(x)

        def step(layer=layer, x=x, dy=dy, res=res, y=y, dx=dx):
            layer.take_weight()
            layer.forward(x, res, y)
            L.demo_dropout(layer.drop, y, y, residual=res)
            layer.grad.zero_()
            layer.backward(dy, dx)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        made.append((graph, step, x, (y, dx, layer.grad)))
    for rep in range(4):
        for graph, step, x, outs in made:
            x.copy_(normal(torch, 100 + rep, *x.shape, dtype=x.dtype))
            step()
            want = [o.clone() for o in outs]
            for o in outs:
                o.fill_(7.0)
            torch.cuda.synchronize()
            graph.replay()
            if rep % 2:
                torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
    made[0][0].replay()  # both in flight
    made[1][0].replay()
    torch.cuda.synchronize()


def test_calls_from_two_threads_on_their_own_streams(torch):
    shapes = ((300, 500, 4000), (64, 2048, 2048))
    results, errors = {}, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                m, n, k = shapes[i]
                x = normal(torch, 50 + i, m, k, dtype=torch.bfloat16)
                w = normal(torch, 60 + i, n, k, std=0.05)
                layer = Layer(torch, w, None, m, torch.zeros_like(w))
                y = torch.empty(m, n, device="cuda")
                for _ in range(5):
                    layer.take_weight()
                    layer.forward(x, None, y)
                s.synchronize()
                results[i] = (y, x, w)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors, errors
    for y, x, w in results.values():
        check_product(torch, y, F.value(*F.quantize(host(x), 0, 0)), F.value(*F.quantize(host(w), 0, 1)))


def test_binding_checks(torch):
    x = torch.zeros(64, 256, device="cuda")
    q = operand(torch, 64, 256)
    d = L.Dropout()
    with pytest.raises(ValueError, match="contiguous"):
        L.demo_dropout(d, x.t(), x.t())
    with pytest.raises(TypeError, match="expected"):
        L.demo_dropout(d, x, x.half())
    with pytest.raises(ValueError, match="elements"):
        L.demo_dropout(d, x, x[:32].contiguous())
    with pytest.raises(ValueError, match="elements"):
        L.demo_dropout(d, x, torch.empty_like(x), residual=x[:1].contiguous())
    with pytest.raises(ValueError, match="neighbouring"):
        L.demo_block_quantize(L.Block(), x.t(), operand(torch, 256, 64))
    with pytest.raises(ValueError, match="overlap"):
        L.demo_block_quantize(L.Block(), x[:1].expand(64, 256), q)
    with pytest.raises(ValueError, match="matrix"):
        L.demo_block_quantize(L.Block(), x.view(-1), q)
    with pytest.raises(ValueError, match="bytes"):
        L.demo_block_quantize(L.Block(), x, q[:-256])
    c = torch.empty(64, 64, device="cuda")
    with pytest.raises(ValueError, match="bytes"):
        L.demo_block_matmul(L.Product(), 64, 64, 512, q, q, c)
    with pytest.raises(ValueError, match="matrix"):
        L.demo_block_matmul(L.Product(), 64, 65, 256, q, operand(torch, 65, 256), c)
    with pytest.raises(TypeError, match="expected"):
        L.demo_block_matmul(L.Product(), 64, 64, 256, q, q, c, addend=c.half())
    with pytest.raises(L.DemoError):
        L.demo_block_matmul(L.Product(fmt_a=5), 64, 64, 256, q, q, c)
    with pytest.raises(L.DemoError):
        L.demo_dropout(L.Dropout(p=2.0), x, x)
    with pytest.raises(L.DemoError):
        L.demo_dropout(d, x[:0], x[:0])


# ------------------------------------------------- precision of the products --

def planted(m, n, k, big, small_a, small_b):
    """One group of eight neighbours in each block of 128: big * big, -big * big
    and a product of +-1 to +-4 times small_a small_b.  Every other product is
    zero, so the result is the sum of the last ones, to the bit."""
    rng = np.random.default_rng(m + n + k)
    va, vb = np.zeros((m, k)), np.zeros((n, k))
    for b in range(k // 128):
        at = 128 * b + 8 * (b % 16)
        order = rng.permutation(8)[:3]
        va[:, at + order[0]], vb[:, at + order[0]] = big, big
        va[:, at + order[1]], vb[:, at + order[1]] = big, -big
        va[:, at + order[2]] = rng.choice([-2, -1, 1, 2], m) * small_a
        vb[:, at + order[2]] = rng.choice([-2, -1, 1, 2], n) * small_b
    return va, vb


PLANTED = [(1, 300, 640), (2, 300, 640), (5, 200, 1280), (16, 77, 1280), (16, 4100, 128),  # one and two rows, few rows
           (70, 130, 640), (512, 500, 8192), (33, 64, 1 << 16),                          # tiles of 64, split too
           (1000, 5000, 256), (1800, 1900, 16512),                                        # of 128, split too
           (2000, 8000, 384), (2040, 8184, 1152)]                                          # of 256


@pytest.mark.parametrize("out", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k", [s for s in PLANTED if s[2] <= 8192])
def test_product_in_16_bits_keeps_13_places(torch, m, n, k, out):
    """1 - 1 + 2^-13 s: the results are at most 4 k / 128 of 2^-13, which both types hold."""
    assert 4 * k // 128 <= 256
    va, vb = planted(m, n, k, 1.0, 2.0**-6, 2.0**-7)
    a, b = (torch.from_numpy(F.pack(v, np.zeros((len(v), -(-k // 128)), np.int64), 0)).cuda() for v in (va, vb))
    c = torch.full((m, n), float("nan"), dtype=dt(torch, out), device="cuda")
    L.demo_block_matmul(L.Product(), m, n, k, a, b, c, workspace=workspace(torch, m, n, k))
    want = torch.from_numpy(va).cuda() @ torch.from_numpy(vb).cuda().t().contiguous()
    assert (want != 0).any() and torch.equal(c.double(), want)


@pytest.mark.parametrize("outliers", [False, True])
@pytest.mark.parametrize("m,n,k", [(16, 64, 2048), (48, 64, 2048), (48, 64, 8192)])
def test_product_in_16_bits_error_of_its_sums(torch, m, n, k, outliers):
    """What the 8-bit instructions leave of a sum.  The addend takes the rounded
    result away, so the call returns what is below that rounding.
    Each product loses what it has below 2^-13 of 2^(the largest sum of two
    codes' exponents in its group of 8): the loss of a sum is at most the sum of
    these remainders, and with their random signs the root of the sum of their
    squares (1.5 times it, over 1024 results and more, is 30 standard deviations).
    On such data that is less than 2^-14 of the results' root mean square."""
    g = torch.Generator().manual_seed(k + m)
    x, w = torch.randn(m, k, generator=g), torch.randn(n, k, generator=g) * 0.02
    if outliers:
        x *= torch.where(torch.rand(k, generator=g) < 0.004, 20.0, 1.0)
    ops, values, parts = [], [], []
    for v, tile in ((x, 0), (w, 1)):
        codes, e = F.quantize(v.numpy(), 0, tile)
        ops.append(torch.from_numpy(F.pack(codes, e, 0)).cuda())
        values.append(torch.from_numpy(F.value(codes, e)).cuda())
        low = np.maximum(np.frexp(codes)[1] - 1, -6)  # exponents of the codes
        power = np.repeat(e, 128, 1)[:, :k] + low
        parts.append(torch.from_numpy(np.where(codes == 0, -10**6, power)).cuda().double().view(len(v), k // 8, 8))
    want = values[0] @ values[1].t().contiguous()
    total = values[0].abs() @ values[1].abs().t().contiguous()
    worst, square = torch.zeros_like(want), torch.zeros_like(want)
    va, vb = values[0].view(m, k // 8, 8), values[1].view(n, k // 8, 8)
    for i in range(m):
        p = (va[i] * vb).abs()
        q = torch.exp2((parts[0][i] + parts[1]).amax(2, keepdim=True).clamp(min=-500) - 13)
        rest = p - torch.floor(p / q) * q
        worst[i], square[i] = rest.sum((1, 2)), (rest * rest).sum((1, 2))
    near = want.to(torch.float16)
    c = torch.empty(m, n, dtype=torch.float16, device="cuda")
    L.demo_block_matmul(L.Product(), m, n, k, *ops, c, addend=-near, workspace=workspace(torch, m, n, k))
    err = c.double() - (want - near.double())
    sums = (17 * (k // 128) + 64) * 2.0**-23 * total + 2.0**-23 * want.abs()
    last = 2.0**-11 * (want - near.double()).abs() * 1.1 + 2.0**-25
    assert (err.abs() <= worst + sums + last * 1.1).all()
    rms = lambda t: float(t.pow(2).mean().sqrt())  # noqa: E731
    assert rms(err) <= 1.5 * float(square.mean().sqrt()) + rms(sums) * 0.05 + rms(last)
    assert rms(err) <= 2.0**-14 * rms(want)
    print(f"rms of the sums' error {rms(err) / rms(want):.2e} of the result, modelled {float(square.mean().sqrt()) / rms(want):.2e}")


@pytest.mark.parametrize("out", ["bf16", "f16"])
def test_product_in_16_bits_is_the_same_every_time(torch, out):
    for m, n, k in ((1, 512, 4096), (9, 512, 4096), (512, 512, 8192), (300, 200, 1000), (2048, 2048, 1024), (2500, 1100, 256), (2000, 8000, 300)):
        a, _, b, _ = operands(torch, m, n, k)
        ws = workspace(torch, m, n, k)
        c = [torch.empty(m, n, dtype=dt(torch, out), device="cuda") for _ in range(3)]
        for x in c:
            L.demo_block_matmul(L.Product(), m, n, k, a, b, x, workspace=ws)
        assert torch.equal(c[0], c[1]) and torch.equal(c[0], c[2])


@pytest.mark.parametrize("m,n,k", PLANTED)
def test_product_in_fp32_keeps_what_8_bit_instructions_lose(torch, m, n, k):
    """448^2 - 448^2 + 2^-4 s: a sum kept to 2^-13 of 448^2 has none of it; 24
    bits hold it (|448^2| < 2^18, everything a multiple of 2^-4)."""
    va, vb = planted(m, n, k, 448.0, 0.25, 0.25)
    a, b = (torch.from_numpy(F.pack(v, np.zeros((len(v), -(-k // 128)), np.int64), 0)).cuda() for v in (va, vb))
    c = torch.full((m, n), float("nan"), device="cuda")
    L.demo_block_matmul(L.Product(), m, n, k, a, b, c, workspace=workspace(torch, m, n, k))
    want = torch.from_numpy(va).cuda() @ torch.from_numpy(vb).cuda().t().contiguous()
    assert 13 + np.log2(0.25**2) < np.log2(448.0**2)  # lost at 13 places
    assert (want != 0).any() and torch.equal(c.double(), want)


@pytest.mark.parametrize("out", ["bf16", "f16"])
@pytest.mark.parametrize("m", [1, 16, 40])
def test_product_range_of_scales_in_16_bits(torch, m, out):
    """Scale bytes far from 1, zero rows, overflow of the type, NaN codes."""
    n, k = 48, 256
    rng = np.random.default_rng(0)
    va, vb = F.round_to(rng.standard_normal((m, k)), 0), F.round_to(rng.standard_normal((n, k)), 0)
    ea, eb = np.zeros((m, 2), np.int64), np.zeros((n, 2), np.int64)
    ea[0], eb[0] = 60, -60
    eb[1] = 30
    eb[3] = -20
    eb[4, 0], eb[4, 1] = 20, -20
    vb[5], eb[5] = 0, -127
    if m > 5:
        ea[1], ea[4, 0], ea[4, 1] = -60, 20, -20
        va[2], ea[2] = 0, -127
    a, b = F.pack(va, ea, 0), F.pack(vb, eb, 0)
    pitch = F.layout(m, k)[0]
    if m > 7:
        a[7 * pitch + 130] = 0x7F
    b[9 * pitch + 5] = 0xFF
    c = torch.empty(m, n, dtype=dt(torch, out), device="cuda")
    L.demo_block_matmul(L.Product(), m, n, k, torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda(), c,
                        workspace=workspace(torch, m, n, k))
    want_nan = torch.zeros(m, n, dtype=torch.bool)
    want_nan[7:8], want_nan[:, 9] = True, True
    assert torch.equal(torch.isnan(c.cpu()), want_nan)
    rows, cols = [i for i in range(m) if i != 7], [j for j in range(n) if j != 9]
    check_product(torch, c.cpu()[rows][:, cols], F.value(va, ea)[rows], F.value(vb, eb)[cols])


# ------------------------------------------------ quantiser, 16-bit sources --

def edges_of_16_bits(torch, dtype):
    """Rows of 256 columns: block maxima next to powers of two and to 1.75
    times one over the type's whole range, in either half of a pair, with
    values below them down to what underflows; subnormals only; the type's
    largest and smallest values; zeros of both signs."""
    f = torch.finfo(dtype)
    low, top, eps = int(np.log2(f.tiny)) + int(np.log2(f.eps)), int(np.floor(np.log2(f.max))), f.eps
    rows = []
    for e in sorted({low, low + 1, low + 3, low - int(np.log2(eps)) - 1, low - int(np.log2(eps)), -9, -1, 0, 8, 9, top - 1, top}):
        for i, m in enumerate((1.0, 1.0 + eps, 1.75, 1.75 + eps, 2.0 - eps)):
            x = np.ldexp(m, e)
            row = np.array([x * 2.0**-j * s for j in range(64) for s in (1, -0.75)] * 2)
            row[128:] *= -1
            rows.append(np.roll(row, i))
    sub = np.arange(256.0) % 120 + 1  # whole multiples of the smallest subnormal
    rows += [sub * 2.0**low, -sub[::-1] * 2.0**low * (np.arange(256) % 2), np.zeros(256), -np.zeros(256)]
    for at, v in ((0, f.max), (1, -f.max), (254, 2.0**low), (255, -(2.0**low))):
        row = np.zeros(256)
        row[at] = row[(at + 128) % 256] = v
        rows.append(row)
    return torch.from_numpy(np.array(rows)).to(dtype).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("tile", [0, 1])
@pytest.mark.parametrize("cols", [256, 251])
def test_quantize_edges_of_16_bit_types(torch, dtype, fmt, tile, cols):
    x = edges_of_16_bits(torch, dt(torch, dtype))[:, :cols].contiguous()
    x = torch.cat([x, x.flip(0)])  # more than one square down
    q, qt = operand(torch, *x.shape), operand(torch, x.shape[1], x.shape[0])
    L.demo_block_quantize(L.Block(fmt=fmt, tile=tile), x, q, qt)
    check_operand(torch, q, host(x), fmt, tile)
    check_operand(torch, qt, host(x).T, fmt, tile)
    small = x[: x.shape[0] // 2] * 0  # nothing but subnormals in a whole square
    small[::3] = x[x.shape[0] // 2 - 8]
    q, qt = operand(torch, *small.shape), operand(torch, small.shape[1], small.shape[0])
    L.demo_block_quantize(L.Block(fmt=fmt, tile=tile), small, q, qt)
    check_operand(torch, q, host(small), fmt, tile)
    check_operand(torch, qt, host(small).T, fmt, tile)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("tile", [0, 1])
@pytest.mark.parametrize("cols", [304, 301])
def test_quantize_infinities_and_nan_of_16_bit_types(torch, dtype, fmt, tile, cols):
    x = normal(torch, 9, 200, cols, dtype=dt(torch, dtype))
    inf, nan = float("inf"), float("nan")
    x[3, 5], x[3, 200], x[150, 20], x[199, cols - 1], x[150, 21], x[151, 20] = inf, nan, -inf, nan, inf, -nan
    x[7] = nan  # blocks of nothing but NaN, and of nothing but infinities
    x[8, :128], x[9, 128:256] = inf, -inf
    x[:128, 40], x[128:, 41] = nan, inf
    x[20, ::2], x[21, 1::2] = nan, inf
    q, qt = operand(torch, 200, cols), operand(torch, cols, 200)
    L.demo_block_quantize(L.Block(fmt=fmt, tile=tile), x, q, qt)
    check_operand(torch, q, host(x), fmt, tile)
    check_operand(torch, qt, host(x).T, fmt, tile)
    x[:128, :128] = nan  # a whole square
    L.demo_block_quantize(L.Block(fmt=fmt, tile=tile), x, q, qt)
    check_operand(torch, q, host(x), fmt, tile)
    check_operand(torch, qt, host(x).T, fmt, tile)


@pytest.mark.parametrize("p", [0.0, 0.2, 1.0 - 2.0**-16, 1.0])
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("tile", [0, 1])
@pytest.mark.parametrize("rows,cols", [(130, 256), (129, 131), (3, 5)])
def test_quantize_to_e4m3_with_dropout(torch, rows, cols, tile, dtype, p):
    """As test_quantize_with_dropout and its range's end, in the other format."""
    x = normal(torch, 10, rows, cols, dtype=dt(torch, dtype))
    top = torch.finfo(x.dtype).max
    x[0, 0] = float("nan")
    x[1::9, ::5] = top
    x[2::9, 1::7] = -top / 1.99
    x[2, 4] = float("inf")
    x[5::9] *= torch.finfo(x.dtype).tiny
    kw = dict(p=p, seed=77, step=3, site=2, chunk_offset=9)
    q, qt = operand(torch, rows, cols), operand(torch, cols, rows)
    L.demo_block_quantize(L.Block(fmt=0, tile=tile), x, q, qt, dropout=L.Dropout(**kw))
    with np.errstate(over="ignore", invalid="ignore"):
        g = np.float32(host(x)) * np.float32(F.scale(p))  # fp32, rounded once
    g = np.where(F.keep(rows * cols, **kw).reshape(rows, cols), g, np.float32(0))
    check_operand(torch, q, g, 0, tile)
    check_operand(torch, qt, g.T, 0, tile)


def test_two_graphs_at_the_same_time(torch):
    """Two captured layers with workspaces of their own, replayed on two streams
    without a wait between them: every output as the eager run's."""
    made = []
    for i, (tokens, n, k) in enumerate(((512, 512, 2048), (500, 768, 1024))):
        layer = Layer(torch, normal(torch, i, n, k, std=0.05), L.Dropout(p=0.1, seed=i), tokens, torch.zeros(n, k, device="cuda"))
        x, dy = (normal(torch, 10 + i, tokens, c, dtype=torch.bfloat16) for c in (k, n))
        res, y, dx = torch.zeros_like(dy), torch.empty_like(dy), torch.empty_like(x)

        def step(layer=layer, x=x, dy=dy, res=res, y=y, dx=dx):
            layer.take_weight()
            layer.forward(x, res, y)
            layer.grad.zero_()
            layer.backward(dy, dx)

        step()
        torch.cuda.synchronize()
        outs = (y, dx, layer.grad)
        want = [o.clone() for o in outs]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        made.append((graph, torch.cuda.Stream(), outs, want, step))  # step holds what the graph reads
    for rep in range(4):
        for _, _, outs, _, _ in made:
            for o in outs:
                o.fill_(7.0)
        torch.cuda.synchronize()
        for _ in range(3):
            for graph, stream, _, _, _ in made:
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for _, _, outs, want, _ in made:
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), rep


def test_a_captured_dropout_draws_its_step_at_every_replay(torch):
    """The configuration is read when the call is made; the backward pass of
    that step, made later and eagerly, draws the same numbers."""
    n = 5000
    x, d = torch.ones(n, device="cuda"), L.Dropout(p=0.5, seed=4, step=10)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    L.demo_dropout(d, x, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.demo_dropout(d, x, y)
    want = torch.from_numpy(F.keep(n, 0.5, seed=4, step=10)).cuda() * 2.0
    for step in (11, 12, 13):
        d.step = step
        y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want.float())
    d.step = 10
    L.demo_dropout_backward(d, x, dx)
    assert torch.equal(dx, y)
