"""Clipping at an infinite limit: c is 1 for every norm but NaN."""
import pytest

from communication_compressed_optimizer_elt_amd import binding as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    L.lib()
    return torch


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_an_infinite_limit_changes_nothing(torch, dtype):
    """No gradient passes it, one with infinities neither; NaN makes everything NaN, as at any limit."""
    for bad in (None, float("inf"), -float("inf"), float("nan")):
        g = torch.randn(5003, generator=torch.Generator().manual_seed(1)).to(getattr(torch, dtype)).cuda()
        if bad is not None:
            g[70] = bad
        sumsq, norm = torch.empty(1, dtype=torch.float64, device="cuda"), torch.empty(1, device="cuda")
        L.demo_grad_norm([g], sumsq)
        out, same = torch.full((5003,), 9.0, device="cuda"), g.clone()
        L.demo_grad_clip([g], sumsq, float("inf"), dst=[out], norm=norm)
        L.demo_grad_clip([same], sumsq, float("inf"))
        if bad is not None and bad != bad:
            assert out.isnan().all() and same.isnan().all() and norm.isnan().all()
        else:
            assert torch.equal(out, g.float()) and torch.equal(same, g)
            assert float(norm) == (float("inf") if bad else pytest.approx(float((g.double() ** 2).sum()) ** 0.5, rel=1e-6))
