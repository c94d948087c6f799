"""The example of state space blocks: its output and every gradient against the same network in 64-bit torch on the
CPU (autograd), and its generation, prompt and captured tokens, against the whole sequence."""
import importlib.util
import os
import sys
from dataclasses import fields

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import depthwise_convolution_nhwc_gb300 as dwc
    dwc.build()
    spec = importlib.util.spec_from_file_location("state_space_blocks", os.path.join(ROOT, "examples", "state_space_blocks.py"))
    m = importlib.util.module_from_spec(spec)
    sys.modules["state_space_blocks"] = m
    spec.loader.exec_module(m)
    return m


def network(z, params, eps):
    """The same in 64-bit torch, position by position."""
    rms = lambda t: t * torch.rsqrt(t.square().mean(-1, keepdim=True) + eps)  # noqa: E731
    silu = lambda t: t * torch.sigmoid(t)  # noqa: E731
    y = rms(z)
    for p in params:
        inner, states = p.A.shape
        taps = p.conv.shape[0]
        h = y @ p.w_in
        line = torch.cat((torch.zeros_like(h[:, :taps - 1, :inner]), h[..., :inner]), 1)
        c = silu(p.conv_bias + sum(p.conv[k] * line[:, k:k + h.shape[1]] for k in range(taps)))
        proj = c @ p.w_x
        delta = torch.log1p(torch.exp(proj[..., :inner] + p.dt_bias))
        state, rows = torch.zeros(z.shape[0], inner, states, dtype=z.dtype), []
        for t in range(z.shape[1]):
            B, C = proj[:, t, None, inner:inner + states], proj[:, t, None, inner + states:]
            state = torch.exp(delta[:, t, :, None] * p.A) * state + (delta[:, t] * c[:, t])[..., None] * B
            rows.append((state * C).sum(-1) + p.D * c[:, t])
        b = (torch.stack(rows, 1) * silu(h[..., inner:])) @ p.w_out
        z = z + p.scale * rms(b) * p.gamma_post
        y = rms(z) * p.gamma_pre
    return y


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,inner,states,taps", [((2, 21, 24), 40, 16, 4), ((3, 35, 16), 32, 5, 3)])
def test_gradients_of_the_network(example, shape, inner, states, taps, dtype):
    """Tolerances: relative 2-norms.  fp32: sums of up to 96 products and about 60 further operations a block, each
    2^-24, through two blocks: (96 + 60) * 2 * 2^-24 = 2e-5, times 5 for the conditioning of norms and gates.  bf16: each of
    about 20 tensors on the way from the input to a gradient and back is rounded with 2^-8 at most (2^-9.5 in the mean
    square): sqrt(40) * 2^-8 = 2.5e-2, taken twice."""
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    params = example.make_params(2, shape[-1], inner, states, taps, dt, seed=3)
    gen = torch.Generator().manual_seed(2)
    z, dy = torch.randn(*shape, generator=gen), torch.randn(*shape, generator=gen).to(dt)
    # (products of fp32 matrices in fp32, not in fewer bits)
    assert torch.get_float32_matmul_precision() == "highest"
    y, _, saved = example.forward(z.cuda(), params)
    dz, grads = example.backward(dy.cuda(), saved, params)
    leaf = lambda t: t.detach().double().cpu().requires_grad_()  # noqa: E731
    zr = leaf(z)
    ref = [example.Block(*(leaf(getattr(p, f.name)) for f in fields(p))) for p in params]
    out = network(zr, ref, example.EPS)
    out.backward(dy.double())
    tol = 1e-4 if dtype == "f32" else 5e-2
    pairs = [("y", y, out.detach()), ("dz", dz, zr.grad)]
    pairs += [(f"{f.name} {i}", getattr(grads[i], f.name), getattr(ref[i], f.name).grad) for i in range(2) for f in fields(ref[i])]
    for name, got, want in pairs:
        assert got.shape == want.shape, name
        off = float((got.double().cpu() - want).norm() / want.norm())
        assert off <= tol, (name, off)


def test_generation_is_the_whole_sequence(example):
    """Outputs of the captured tokens against one pass over prompt and tokens (fp32; the same operations in another order:
    the tolerance of the gradients' test)."""
    params = example.make_params(2, 32, 64, 16, 4, torch.float32, seed=1)
    z = torch.randn(3, 19, 32, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    out = example.generate(z, params, 6)
    y, _, _ = example.forward(z, params)
    whole, _, _ = example.forward(torch.cat((z, y[:, -1:].float(), out[:, :-1]), 1), params)
    assert float((out - whole[:, 19:]).norm() / out.norm()) <= 1e-4


def test_training_runs(example):
    params = example.make_params(2, 32, 64, 16, 4, torch.bfloat16)
    gen = torch.Generator(device="cuda").manual_seed(1)
    z, target = (torch.randn(2, 40, 32, generator=gen, device="cuda") for _ in range(2))
    for _ in range(3):
        assert torch.isfinite(example.train_step(z, target, params, rate=0.5))
