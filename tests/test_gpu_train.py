"""The operators around the linear layer as a training step runs them: norm with
the residual, 8-bit or 4-bit products, the backward pass, the gradient's norm,
clipping into the flat gradient and the optimizer step's encode, eager and
captured."""
import linear_forms as F
import numpy as np
import pytest
import train_forms as T

from communication_compressed_optimizer_elt_amd import binding as L

pytestmark = pytest.mark.gpu
M, N, K = 200, 144, 256  # tokens, outputs, width


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


class Step:
    """One block: h = residual + x, y = norm(h), z = y W^T; and all of its gradients."""

    def __init__(self, torch, four_bits):
        byte = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        layout = L.demo_mx_layout if four_bits else L.demo_block_layout
        buf = lambda r, c: byte(layout(r, c)["total_bytes"])  # noqa: E731
        self.four = four_bits
        self.x, self.res, self.dz = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((M, K), (M, K), (M, N)))
        self.dh = torch.empty_like(self.x)
        self.theta = torch.empty(N * K + K, device="cuda")  # W, then the norm's weight
        self.w, self.g = self.theta[: N * K].view(N, K), self.theta[N * K:]
        self.h, self.y, self.z = torch.empty_like(self.x), torch.empty_like(self.x), torch.empty_like(self.dz)
        self.rstd = torch.empty(M, device="cuda")
        self.yq, self.yt, self.wq, self.wt = buf(M, K), buf(K, M), buf(N, K), buf(K, N)
        self.gq, self.gt = buf(M, N), buf(N, M)
        self.dy, self.dx = torch.empty_like(self.x), torch.empty_like(self.x)
        self.dw, self.dg = torch.empty(N, K, device="cuda"), torch.empty(K, device="cuda")
        self.flat = torch.empty(N * K + K, device="cuda")
        self.sumsq, self.norm = torch.empty(1, dtype=torch.float64, device="cuda"), torch.empty(1, device="cuda")
        self.work = byte(L.BLOCK_MAX_WORKSPACE)
        self.grads = L.Tensors([self.dw, self.dg])
        self.places = L.Tensors(self.flat.split([N * K, K]))
        self.opt = L.Config(scheme=L.SCHEME_DCT, k=4)
        self.mom = torch.empty_like(self.flat)
        self.payload = byte(L.demo_payload_layout(self.opt, self.flat.numel())["total_bytes"])
        self.q = torch.empty_like(self.flat)

    def fill(self, torch, seed):
        for i, (t, std) in enumerate(((self.x, 1), (self.res, 2), (self.dz, 0.1), (self.dh, 0.1), (self.theta, 0.1), (self.mom, 0.01))):
            t.copy_(normal(torch, seed + i, *t.shape, std=std))
        self.g.add_(1.0)

    def run(self):
        norm = L.Norm(eps=1e-5)
        if self.four:
            cfg = back = L.Mx()
            L.demo_mx_quantize(L.Mx(tile=1), self.w, self.wq, self.wt)
            L.demo_rms_norm(norm, self.x, self.g, residual=self.res, h=self.h, y=self.y, rstd=self.rstd)
            L.demo_mx_quantize(cfg, self.y, self.yq, self.yt)
            L.demo_mx_quantize(cfg, self.dz, self.gq, self.gt)
            mul = L.demo_mx_matmul
        else:
            cfg, back = L.Product(), L.Product(fmt_a=L.FMT_E5M2)
            L.demo_block_quantize(L.Block(tile=1), self.w, self.wq, self.wt)
            L.demo_rms_norm(norm, self.x, self.g, residual=self.res, h=self.h, rstd=self.rstd, operand=self.yq, operand_t=self.yt)
            L.demo_block_quantize(L.Block(fmt=L.FMT_E5M2), self.dz, self.gq, self.gt)
            mul = L.demo_block_matmul
        mul(cfg, M, N, K, self.yq, self.wq, self.z, workspace=self.work)
        mul(back, M, K, N, self.gq, self.wt, self.dy, workspace=self.work)
        mul(back, N, K, M, self.gt, self.yt, self.dw, workspace=self.work)
        L.demo_rms_norm_backward(norm, self.dy, self.h, self.g, self.rstd, self.dx, dresidual=self.dh, dweight=self.dg, workspace=self.work)
        L.demo_grad_norm(self.grads, self.sumsq, workspace=self.work)
        L.demo_grad_clip(self.grads, self.sumsq, 0.5, dst=self.places, norm=self.norm)
        L.demo_encode(self.opt, self.flat.numel(), self.flat, self.mom, self.payload, self.q)

    def outputs(self):
        return {n: getattr(self, n).clone() for n in ("h", "z", "dx", "dw", "dg", "flat", "norm", "mom", "q", "payload")}


@pytest.mark.parametrize("four", [False, True])
def test_step_against_64_bits(torch, four):
    """Quantisation is the step's own; beside it every gradient is within a
    hundredth of the 64-bit chain on the values that the operands hold."""
    s = Step(torch, four)
    s.fill(torch, 10)
    mom = host(s.mom)
    s.run()
    h = host((s.x.float() + s.res.float()).bfloat16())
    r, y = T.norm(h, host(s.g), 1e-5)
    if four:
        y = host(s.y)  # what is quantised is the rounded y
        v = lambda x, tile=0, fmt=0: T.mx_value(*T.mx_quantize(x, tile))  # noqa: E731
    else:
        v = lambda x, tile=0, fmt=0: F.value(*F.quantize(x, fmt, tile))  # noqa: E731
    z = v(y) @ v(host(s.w), 1).T
    dz = host(s.dz)
    dy = v(dz, 0, 1) @ v(host(s.w).T, 1).T
    dw = v(dz.T, 0, 1) @ v(y.T).T
    dx, dg, _, _ = T.norm_backward(dy, h, host(s.g), r, host(s.dh))
    norm = ((dw**2).sum() + (dg**2).sum()) ** 0.5
    flat = np.concatenate([dw.reshape(-1), dg]) * min(1.0, 0.5 / (norm + 1e-6))
    for got, want in ((s.z, z), (s.dx, dx), (s.dw, dw), (s.dg, dg), (s.flat, flat), (s.norm, np.array([norm]))):
        assert np.linalg.norm(host(got) - want) <= 0.01 * np.linalg.norm(want)
    assert norm > 0.5  # it was clipped
    u = np.float32(0.9).astype(np.float64) * mom + host(s.flat)  # momentum and what was sent make u again
    assert np.abs(host(s.mom) + host(s.q) - u).max() <= 1e-5 * np.abs(u).max()


@pytest.mark.parametrize("four", [False, True])
def test_captured_step(torch, four):
    """A captured step replays with new inputs, beside another captured step on a stream of its own."""
    eager, steps = Step(torch, four), [Step(torch, four) for _ in range(2)]
    graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for s, stream in zip(steps, streams):
        s.fill(torch, 1)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            s.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            s.run()
        graphs.append(g)
    for seed in (100, 200, 300):
        for i, s in enumerate(steps):
            s.fill(torch, seed + 50 * i)
        torch.cuda.synchronize()
        for g, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
        torch.cuda.synchronize()
        for i, s in enumerate(steps):
            eager.fill(torch, seed + 50 * i)
            eager.run()
            want, got = eager.outputs(), s.outputs()
            assert all(torch.equal(want[n], got[n]) for n in want), [n for n in want if not torch.equal(want[n], got[n])]
