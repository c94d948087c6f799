"""The example of depthwise residual blocks: its output and every gradient against the same network in
64-bit torch on the CPU (autograd), with the dropout masks of the fp64 definition, and the fall of
its loss."""
import importlib.util
import os

import numpy as np
import pytest
import torch
import torch.nn.functional as F

from oracle import norm as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import depthwise_convolution_nhwc_gb300 as dwc
    dwc.build()
    spec = importlib.util.spec_from_file_location("residual_blocks", os.path.join(ROOT, "examples", "residual_blocks.py"))
    m = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["residual_blocks"] = m
    spec.loader.exec_module(m)
    return m


def masks(shape, p, seed, offset):
    q = np.floor(p * 65536 + 0.5) / 65536
    keep = ref.kept(0, int(np.prod(shape)), p, seed, offset).reshape(shape)
    return torch.from_numpy(keep / (1 - q))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,taps", [((2, 9, 7, 40), 3), ((1, 14, 14, 72), 7), ((2, 6, 5, 33), 5)])
def test_gradients_of_the_network(example, shape, taps, dtype):
    """Tolerances: relative 2-norms.  fp32: the convolutions' 1e-5 (of the sum of absolute products, so less of
    the norm) and a few 1e-7 of the norms, over three blocks: 1e-4.  bf16: each of the about 12 tensors
    on the way from the input to a gradient is rounded with u = 2^-8 at most (2^-9.5 in the mean square),
    and the residual stream carries them on without growth: sqrt(12) * 2^-8 = 1.4e-2, taken twice."""
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    p, seed, step, blocks = 0.25, 77, 3, 3
    params = example.make_params(blocks, taps, shape[-1], dt, seed=5)
    gen = torch.Generator().manual_seed(2)
    for i in range(blocks + 1):
        params.gamma[i] += 0.2 * torch.randn(shape[-1], generator=gen).cuda()
        params.beta[i] += 0.2 * torch.randn(shape[-1], generator=gen).cuda()
    x, dy = torch.randn(*shape, generator=gen), torch.randn(*shape, generator=gen).to(dt)
    y, saved = example.forward(x.cuda(), params, p, seed, step)
    dx, grads = example.backward(dy.cuda(), saved, params, p, seed, step)

    leaf = lambda t: t.detach().double().cpu().requires_grad_()  # noqa: E731
    xr, w = leaf(x), [leaf(t) for t in params.w]
    gamma, beta = [leaf(t) for t in params.gamma], [leaf(t) for t in params.beta]
    base = step * (blocks + 1)
    z = xr * masks(shape, p, seed, base)
    norm = lambda z, i: F.layer_norm(z, (shape[-1],), gamma[i], beta[i], example.EPS)  # noqa: E731
    out = norm(z, 0)
    for i in range(blocks):
        k = w[i].permute(2, 0, 1).unsqueeze(1)
        b = F.conv2d(out.permute(0, 3, 1, 2), k, padding=taps // 2, groups=shape[-1]).permute(0, 2, 3, 1)
        z = z + b * masks(shape, p, seed, base + i + 1)
        out = norm(z, i + 1)
    out.backward(dy.double())
    tol = 1e-4 if dtype == "f32" else 2.8e-2
    pairs = [("y", y, out.detach()), ("dx", dx, xr.grad)]
    pairs += [(f"dw{i}", grads.w[i], w[i].grad) for i in range(blocks)]
    pairs += [(f"dgamma{i}", grads.gamma[i], gamma[i].grad) for i in range(blocks + 1)]
    pairs += [(f"dbeta{i}", grads.beta[i], beta[i].grad) for i in range(blocks + 1)]
    for name, got, want in pairs:
        off = float((got.double().cpu() - want).norm() / want.norm())
        assert off <= tol, (name, off)


def test_loss_falls(example):
    params = example.make_params(2, 3, 64, torch.bfloat16)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, target = (torch.randn(2, 8, 8, 64, generator=gen, device="cuda") for _ in range(2))
    losses = [float(example.train_step(x, target, params, 0.1, 9, k, rate=0.02 * 64)) for k in range(12)]
    assert losses[-1] < losses[0] and all(np.isfinite(losses))
