"""Where fp32's range ends inside the norm and the 4-bit product, as documented."""
import numpy as np
import pytest
import train_forms as T

from communication_compressed_optimizer_elt_amd import binding as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    L.lib()
    return torch


@pytest.mark.parametrize("cols", [8, 64, 520, 4096, 9000])
def test_norm_of_tiny_rows(torch, cols):
    """eps 0.  From 2^-63 on squares are normal: r to 36 roundings of 2^-24.  Magnitudes of 2^-75 and
    less have no square: r is infinite, and so is y.  Any eps that fp32 holds as a normal number is
    larger than what is lost."""
    w = torch.ones(cols, device="cuda")
    x = torch.empty(4, cols, device="cuda")
    x[0], x[1], x[2], x[3] = 1.37 * 2.0**-63, 2.0**-75, -1.5 * 2.0**-100, 2.0**-126
    y, r = torch.empty_like(x), torch.empty(4, device="cuda")
    L.demo_rms_norm(L.Norm(eps=0.0), x, w, y=y, rstd=r)
    assert abs(float(r[0].double()) * float(x[0, 0].double()) - 1) <= 36 * 2.0**-24
    assert (r[1:] == float("inf")).all()
    assert (y[1] == float("inf")).all() and (y[2] == -float("inf")).all() and (y[3] == float("inf")).all()
    eps = 2.0**-126
    L.demo_rms_norm(L.Norm(eps=eps), x, w, y=y, rstd=r)
    want = 1 / ((x.double() ** 2).mean(1) + eps).sqrt()
    assert ((r.double() / want - 1).abs() <= 36 * 2.0**-24).all()


# (1) and (2) rows, few rows, tiles of 64, 128 and 256, and 256 of workgroups that stay
SIZES = [(1, 64, 256), (2, 64, 300), (8, 64, 256), (70, 80, 256), (2300, 2101, 256), (4100, 2061, 300), (4100, 2064, 1024)]


def product(torch, m, n, k, ea, eb):
    g = np.random.default_rng(1)
    grid, kb = np.concatenate([T.GRID, -T.GRID]), -(-k // 32)
    ca, cb, ea, eb = g.choice(grid, (m, k)), g.choice(grid, (n, k)), np.full((m, kb), ea), np.full((n, kb), eb)
    c = torch.empty(m, n, device="cuda")
    ws = torch.empty(max(L.demo_mx_workspace(L.Mx(), m, n, k), 16), dtype=torch.uint8, device="cuda")
    L.demo_mx_matmul(L.Mx(), m, n, k, torch.from_numpy(T.mx_pack(ca, ea)).cuda(), torch.from_numpy(T.mx_pack(cb, eb)).cuda(), c, workspace=ws)
    a, b = (torch.from_numpy(T.mx_value(*x)).cuda() for x in ((ca, ea), (cb, eb)))
    return c, a @ b.t().contiguous(), a.abs() @ b.abs().t().contiguous()


@pytest.mark.parametrize("m,n,k", SIZES)
def test_products_of_the_smallest_and_largest_scales(torch, m, n, k):
    """Sums of multiples of 2^-149 below 2^24 of them are exact, whatever the scales that meet."""
    for ea, eb in ((127, -127), (-127, 127), (-127, 0), (-70, -70), (-75, -72), (0, -127)):
        c, want, s = product(torch, m, n, k, ea, eb)
        assert float(s.max()) < 2.0 ** (ea + eb - 2 + 24) and ea + eb - 2 >= -149
        assert torch.equal(c.double(), want)


@pytest.mark.parametrize("m,n,k", SIZES)
def test_products_below_the_smallest_number(torch, m, n, k):
    """Of 128 of the sum a matrix instruction keeps multiples of 2^-149 of 17 parts, as of normal ones 2^-23 of the largest."""
    for ea, eb in ((-127, -22), (-127, -24), (-127, -127)):
        c, want, _ = product(torch, m, n, k, ea, eb)
        assert ((c.double() - want).abs() <= (17 * -(-k // 128) + 64) * 2.0**-149).all()


@pytest.mark.parametrize("m,n,k", SIZES)
def test_products_beyond_the_largest_number(torch, m, n, k):
    """Below the range's end in magnitude all is finite; what passes it is never a finite number."""
    for ea, eb in ((60, 60), (127, -5), (64, 60), (127, 127)):
        c, want, s = product(torch, m, n, k, ea, eb)
        assert c[s < 2.0**127].isfinite().all()
        assert not c[want.abs() >= 2.0**128 * 1.001].isfinite().any()
        one = c.isinf() & (want.abs() < 2.0**128)
        assert (s[one | c.isnan()] >= 2.0**127).all()
