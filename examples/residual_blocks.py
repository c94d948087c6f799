"""A training loop over depthwise residual blocks, forward and backward entirely calls of this library
(the loss and the update of the weights are PyTorch's):

    z_0 = dropout(x),  y_0 = norm(z_0);    b_i = dwc(y_i),  z_{i+1} = z_i + dropout(b_i),
    y_{i+1} = norm(z_{i+1})

Activations are N x H x W x C; the residual stream z is fp32, the branches (y, b and their gradients) fp32 or
bf16.  The add, the dropout and the norm behind it are one call (``add_layer_norm_fwd``); no mask is
stored, the backward pass draws it again from the seed and the offset of its layer and step.

    python examples/residual_blocks.py [--dtype bf16] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir))

import torch  # noqa: E402

import depthwise_convolution_nhwc_gb300 as dwc  # noqa: E402

EPS = 1e-5


@dataclass
class Params:
    """Filters of the blocks (FH x FW x C, branch dtype) and the norms' fp32 weights, one more of these."""
    w: list
    gamma: list
    beta: list


def make_params(blocks: int, taps: int, channels: int, dtype, seed: int = 0) -> Params:
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = [(torch.randn(taps, taps, channels, generator=g, device="cuda") / taps).to(dtype) for _ in range(blocks)]
    return Params(w, [torch.ones(channels, device="cuda") for _ in range(blocks + 1)],
                  [torch.zeros(channels, device="cuda") for _ in range(blocks + 1)])


def forward(x, params: Params, p: float, seed: int, step: int):
    """(output, what the backward pass needs).  Offset (step, layer) counts the dropouts apart."""
    blocks, dtype = len(params.w), params.w[0].dtype
    pad = params.w[0].shape[0] // 2
    base = step * (blocks + 1)
    z = dwc.dropout_fwd(x, p, seed, base)
    y, mean, rstd = dwc.layer_norm_fwd(z, params.gamma[0], params.beta[0], EPS, out_dtype=dtype, stats=True)
    saved = [(z, mean, rstd, y)]
    for i, w in enumerate(params.w):
        b = dwc.fwd(y, w, 1, pad, out_dtype=dtype)
        y, z, mean, rstd = dwc.add_layer_norm_fwd(b, z, params.gamma[i + 1], params.beta[i + 1], EPS, p, seed,
                                                  base + i + 1, stats=True)
        saved.append((z, mean, rstd, y))
    return y, saved


def backward(dy, saved, params: Params, p: float, seed: int, step: int):
    """(dx, gradients in the form of Params) from the gradient of the output."""
    blocks, dtype = len(params.w), params.w[0].dtype
    taps = tuple(params.w[0].shape[:2])
    pad, base = taps[0] // 2, step * (blocks + 1)
    grads = Params([None] * blocks, [None] * (blocks + 1), [None] * (blocks + 1))
    dz = None
    for i in reversed(range(blocks)):
        z, mean, rstd, _ = saved[i + 1]
        db, dz, grads.gamma[i + 1], grads.beta[i + 1] = dwc.add_layer_norm_bwd(
            dy, z, mean, rstd, params.gamma[i + 1], dz, p, seed, base + i + 1)
        y = saved[i][3]
        grads.w[i] = dwc.bwd_filter(y, db, taps, 1, pad)
        dy = dwc.bwd_data(db, params.w[i], y.shape[1:3], 1, pad, out_dtype=dtype)
    z, mean, rstd, _ = saved[0]
    if dy.dtype == z.dtype:    # z_0 = 0 + dropout(x): the residual form's gradient of its branch is dx
        dx, _, grads.gamma[0], grads.beta[0] = dwc.add_layer_norm_bwd(dy, z, mean, rstd, params.gamma[0], dz, p, seed, base)
    else:                      # (that one would be in the branches' type; x is fp32)
        _, dz, grads.gamma[0], grads.beta[0] = dwc.add_layer_norm_bwd(dy, z, mean, rstd, params.gamma[0], dz)
        dx = dwc.dropout_bwd(dz, p, seed, base, out=dz)
    return dx, grads


def train_step(x, target, params: Params, p: float, seed: int, step: int, rate: float):
    """One step of gradient descent on half the mean squared error; the loss as a device tensor."""
    y, saved = forward(x, params, p, seed, step)
    diff = y.float() - target
    _, grads = backward((diff / diff.numel()).to(y.dtype), saved, params, p, seed, step)
    for mine, theirs in ((params.w, grads.w), (params.gamma, grads.gamma), (params.beta, grads.beta)):
        for w, d in zip(mine, theirs):
            w.sub_((rate * d).to(w.dtype))
    return 0.5 * diff.square().mean()


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="bf16")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--blocks", type=int, default=3)
    ap.add_argument("--shape", type=int, nargs=4, default=(8, 28, 28, 256), metavar=("N", "H", "W", "C"))
    ap.add_argument("--taps", type=int, default=7)
    ap.add_argument("--dropout", type=float, default=0.1)
    a = ap.parse_args()
    dtype = torch.float32 if a.dtype == "f32" else torch.bfloat16
    params = make_params(a.blocks, a.taps, a.shape[-1], dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, target = (torch.randn(*a.shape, generator=g, device="cuda") for _ in range(2))
    for step in range(a.steps):
        loss = train_step(x, target, params, a.dropout, 1234, step, rate=0.02 * a.shape[-1])
        if step % 5 == 0 or step == a.steps - 1:
            print(f"step {step:3d}  loss {float(loss):.4f}")


if __name__ == "__main__":
    main()
