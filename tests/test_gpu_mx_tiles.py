"""Products of 4-bit operands in each kind of tile, whole and cut at its edges,
against 64 bits on the GPU: dropouts, NaN blocks, scales far from one, splits, odd
widths, results past the caches.

Tolerances: test_gpu_mx's, (17 ceil(k/128) + 64) 2^-23 S + 2^-23 |result| + u |result|,
S the sum of magnitudes, u half a step of the type.
"""
import functools

import linear_forms as F
import numpy as np
import pytest
import train_forms as T

from communication_compressed_optimizer_elt_amd import binding as L

pytestmark = pytest.mark.gpu
DT = ["float32", "float16", "bfloat16"]

# 128-tiles (306 of them): even and odd widths, cut at both ends; 128-tiles in two splits
# (240 and 65 steps of 256); 256-tiles one a workgroup, of odd width or an odd number of steps;
# 256-tiles of workgroups that stay, unless something is added
TILES = [(2300, 2104, 700), (2300, 2101, 700), (2040, 1797, 16500), (2040, 1800, 16500), (4100, 2061, 700), (4100, 2064, 700),
         (4100, 2064, 1000)]


@pytest.fixture(scope="module")
def torch():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    L.lib()
    return torch


@functools.lru_cache(maxsize=8)
def packed(torch, seed, rows, cols, spread=6, nan=(), exponent=0):
    """(operand, its values on the GPU) of random codes and exponents; nan: (row, block) pairs."""
    g = np.random.default_rng(seed)
    codes = g.choice(np.concatenate([T.GRID, -T.GRID]), (rows, cols))
    e = g.integers(-spread, spread + 1, (rows, -(-cols // 32))) + exponent
    for at in nan:
        e[at] = 128
    return torch.from_numpy(T.mx_pack(codes, e)).cuda(), torch.from_numpy(T.mx_value(codes, e)).cuda()


def workspace(torch, m, n, k):
    return torch.empty(max(L.demo_mx_workspace(L.Mx(), m, n, k), 16), dtype=torch.uint8, device="cuda")


def check_product(torch, c, a, b, addend=None, mask=None, scale=1.0):
    want, s = a @ b.t().contiguous(), a.abs() @ b.abs().t().contiguous()
    f = torch.finfo(c.dtype)
    if mask is not None:
        want, s = want * scale * mask, s * scale * mask
    err = (17 * -(-a.shape[1] // 128) + 64) * 2.0**-23 * s + 2.0**-23 * want.abs()
    if addend is not None:
        want = want + addend.double()
        err = err + 2.0**-23 * (addend.double().abs() + want.abs())
    bound = err + f.eps / 2 * (want.abs() + err) + f.tiny * f.eps / 2
    over = (want.abs() + err >= f.max) & c.isinf() & (c * want > 0)
    assert (over | ((c.double() - want).abs() <= bound)).all()


def test_the_sizes_split(torch):
    assert all(L.demo_mx_workspace(L.Mx(), m, n, k) == (2 * m * n * 4 if k == 16500 else 0) for m, n, k in TILES)


@pytest.mark.parametrize("m,n,k", TILES)
@pytest.mark.parametrize("dtype", DT)
def test_product(torch, m, n, k, dtype):
    (qa, a), (qb, b) = packed(torch, m + n, m, k), packed(torch, n + k, n, k)
    c = torch.full((m + 1, n), 9.0, dtype=getattr(torch, dtype), device="cuda")
    ws = workspace(torch, m, n, k)
    L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, c[:m], workspace=ws)
    assert (c[m] == 9.0).all()
    check_product(torch, c[:m], a, b)
    g = torch.Generator(device="cuda").manual_seed(3)
    add = torch.randn(m, n, generator=g, device="cuda").mul_(10).to(c.dtype)
    acc, other = add.clone(), torch.empty_like(add)
    L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, acc, addend=acc, workspace=ws)
    L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, other, addend=add, workspace=ws)
    assert torch.equal(acc, other)
    check_product(torch, acc, a, b, add)


@pytest.mark.parametrize("m,n,k", TILES)
@pytest.mark.parametrize("dtype", DT)
def test_product_through_a_dropout(torch, m, n, k, dtype):
    (qa, a), (qb, b) = packed(torch, 1, m, k, spread=2), packed(torch, 2, n, k, spread=2)
    kw = dict(p=0.25, seed=9, step=4, site=2, chunk_offset=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    mask = torch.from_numpy(F.keep(m * n, **kw).reshape(m, n)).cuda()
    for add in (None, torch.randn(m, n, generator=g, device="cuda").to(getattr(torch, dtype))):
        c = torch.empty(m, n, dtype=getattr(torch, dtype), device="cuda") if add is None else add.clone()
        L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, c, addend=None if add is None else c, dropout=L.Dropout(**kw),
                         workspace=workspace(torch, m, n, k))
        check_product(torch, c, a, b, add, mask, F.scale(0.25))


@pytest.mark.parametrize("m,n,k", TILES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("add", [False, True])
def test_nan_blocks(torch, m, n, k, dtype, add):
    """A block of scale byte 255 makes its row, or its column, NaN and leaves the others."""
    last = (k + 31) // 32 - 1
    qa, a = packed(torch, 1, m, k, nan=((m - 1, 3), (130, last), (0, 0)))
    qb, b = packed(torch, 2, n, k, nan=((n - 1, last), (129, 0)))
    c = torch.zeros(m, n, dtype=getattr(torch, dtype), device="cuda")
    L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, c, addend=c if add else None, workspace=workspace(torch, m, n, k))
    rows, cols = a.isnan().any(1), b.isnan().any(1)
    assert rows.sum() == 3 and cols.sum() == 2
    assert torch.equal(c.isnan(), rows[:, None] | cols[None, :])
    check_product(torch, c[~rows][:, ~cols], a[~rows], b[~cols])


@pytest.mark.parametrize("m,n,k", TILES)
@pytest.mark.parametrize("dtype", DT)
def test_scales_far_from_one(torch, m, n, k, dtype):
    """Products of large and small blocks that meet in the middle, and zero rows."""
    qa, a = packed(torch, 1, m, k, spread=2, exponent=-118)
    qb, b = packed(torch, 2, n, k, spread=2, exponent=116)
    c = torch.empty(m, n, dtype=getattr(torch, dtype), device="cuda")
    L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, c, workspace=workspace(torch, m, n, k))
    check_product(torch, c, a, b)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("k", [1024, 1500])
def test_results_past_the_caches(torch, dtype, k):
    """Results of more than 96 MiB in each type, several tiles a workgroup, moved back inside at both ends."""
    m, n = 8200, 8200
    assert m * n * 2 > 96 << 20
    (qa, a), (qb, b) = packed(torch, k, m, k), packed(torch, n, n, k)
    c = torch.full((m + 1, n), 9.0, dtype=getattr(torch, dtype), device="cuda")
    L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, c[:m])
    assert (c[m] == 9.0).all()
    check_product(torch, c[:m], a, b)


def test_three_tiles_a_workgroup_repeat(torch):
    """The same bits at every call, with other work between."""
    m, n, k = 8200, 8200, 1024
    (qa, _), (qb, _) = packed(torch, 1, m, k), packed(torch, 2, n, k)
    for dtype in (torch.bfloat16, torch.float32):
        first = torch.empty(m, n, dtype=dtype, device="cuda")
        L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, first)
        for _ in range(3):
            c = torch.zeros_like(first)
            L.demo_mx_matmul(L.Mx(), m, n, k, qa, qb, c)
            assert torch.equal(c, first)
