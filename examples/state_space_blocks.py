"""A training loop and a generation loop over state space blocks; between the projections (plain matrix products) every
operator, forward and backward, is a call of this library:

    y_0 = norm(z_0);   [h, g] = y_i W_in;   c = silu(causal_conv(h));   [dt, B, C] = c W_x
    s = selective_scan(c, dt, A, B, C, D, gate g);   b = s W_out
    z_{i+1} = z_i + scale * norm(b) * gamma_post,   y_{i+1} = norm(z_{i+1}) * gamma_pre

Activations are sequences x positions x width; the residual stream z is fp32, the rest fp32 or bf16.  Generation runs the
prompt through the sequence kernels and then one token at a time from the states that they leave, as a captured graph.

    python examples/state_space_blocks.py [--dtype bf16] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass, fields

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir))

import torch  # noqa: E402

import depthwise_convolution_nhwc_gb300 as dwc  # noqa: E402

EPS = 1e-5


@dataclass
class Block:
    """Matrices in the branches' dtype, everything else fp32."""
    w_in: torch.Tensor       # width x 2 inner
    conv: torch.Tensor       # taps x inner
    conv_bias: torch.Tensor
    w_x: torch.Tensor        # inner x (inner + 2 states)
    A: torch.Tensor          # inner x states
    D: torch.Tensor
    dt_bias: torch.Tensor
    w_out: torch.Tensor      # inner x width
    gamma_post: torch.Tensor
    gamma_pre: torch.Tensor
    scale: torch.Tensor


def make_params(blocks: int, width: int, inner: int, states: int, taps: int, dtype, seed: int = 0) -> list:
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return [Block((r(width, 2 * inner) / width ** 0.5).to(dtype), r(taps, inner) / taps ** 0.5, 0.1 * r(inner),
                  (r(inner, inner + 2 * states) / inner ** 0.5).to(dtype),
                  -torch.arange(1, states + 1, device="cuda") * torch.exp(0.1 * r(inner, states)), 1 + 0.1 * r(inner),
                  r(inner) - 3.0, (r(inner, width) / inner ** 0.5).to(dtype), 1 + 0.1 * r(width), 1 + 0.1 * r(width),
                  0.5 + 0.1 * r(width)) for _ in range(blocks)]


def split(s, p: Block):
    """dt, B and C, as slices of one projection."""
    inner, states = p.A.shape
    return s[..., :inner], s[..., inner:inner + states], s[..., inner + states:]


def first_norm(z, dtype):
    """The norm in front of the first block: a block norm without a branch."""
    return dwc.block_norm_fwd(torch.zeros_like(z, dtype=dtype), z, eps=EPS, stats=True)


def forward(z, params: list):
    """(output, final residual stream, what the backward pass needs)."""
    dtype = params[0].w_in.dtype
    y, z, _, rstd = first_norm(z, dtype)
    saved = [(z, rstd)]
    for p in params:
        inner = p.A.shape[0]
        h = y @ p.w_in
        c = dwc.causal_conv_fwd(h[..., :inner], p.conv, p.conv_bias, "silu")
        proj = c @ p.w_x
        dt, B, C = split(proj, p)
        s, kept = dwc.selective_scan_fwd(c, dt, p.A, B, C, p.D, h[..., inner:], p.dt_bias, save=True)
        b = s @ p.w_out
        y_next, z, post, pre = dwc.block_norm_fwd(b, z, p.gamma_post, p.gamma_pre, None, p.scale, eps=EPS, stats=True)
        saved.append((y, h, c, proj, s, kept, b, z, post, pre))
        y = y_next
    return y, z, saved


def backward(dy, saved, params: list):
    """(dz, gradients in the form of the parameters) from the gradient of the output."""
    flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
    dz, grads = None, [None] * len(params)
    for i in reversed(range(len(params))):
        p = params[i]
        y, h, c, proj, s, kept, b, z, post, pre = saved[i + 1]
        inner = p.A.shape[0]
        db, dz, _, dpost, dpre, dscale = dwc.block_norm_bwd(dy, b, z, post, pre, p.gamma_post, p.gamma_pre, None, p.scale, dz=dz)
        ds = db @ p.w_out.t()
        dt, B, C = split(proj, p)
        du, ddt, dA, dB, dC, dD, dg, dbias, _ = dwc.selective_scan_bwd(ds, c, dt, p.A, B, C, kept, p.D, h[..., inner:], p.dt_bias)
        dproj = torch.cat((ddt, dB, dC), -1)
        dc = torch.addmm(flat(du), flat(dproj), p.w_x.t()).view_as(c)
        dh, dconv, dconv_bias, _ = dwc.causal_conv_bwd(dc, h[..., :inner], p.conv, p.conv_bias, "silu")
        dh = torch.cat((dh, dg), -1)
        grads[i] = Block(flat(y).t() @ flat(dh), dconv, dconv_bias, flat(c).t() @ flat(dproj), dA, dD, dbias, flat(s).t() @ flat(db),
                         dpost, dpre, dscale)
        dy = dh @ p.w_in.t()
    z, rstd = saved[0]
    # the first norm: y = z rstd, its branch zero
    zero = torch.zeros_like(z, dtype=dy.dtype)
    dz = dwc.block_norm_bwd(dy, zero, z, torch.zeros_like(rstd), rstd, dz=dz)[1]
    return dz, grads


def train_step(z, target, params: list, rate: float):
    """One step of gradient descent on half the mean squared error; the loss as a device tensor."""
    y, _, saved = forward(z, params)
    diff = y.float() - target
    _, grads = backward((diff / diff.numel()).to(y.dtype), saved, params)
    for p, g in zip(params, grads):
        for f in fields(p):
            w, d = getattr(p, f.name), getattr(g, f.name)
            w.sub_((rate * d).to(w.dtype))
    return 0.5 * diff.square().mean()


def prompt(z, params: list):
    """(output, the states that a token goes on from)."""
    y = first_norm(z, params[0].w_in.dtype)[0]
    states = []
    for p in params:
        inner = p.A.shape[0]
        h = y @ p.w_in
        c, conv_state = dwc.causal_conv_fwd(h[..., :inner], p.conv, p.conv_bias, "silu", final=True)
        dt, B, C = split(c @ p.w_x, p)
        s, scan_state = dwc.selective_scan_fwd(c, dt, p.A, B, C, p.D, h[..., inner:], p.dt_bias, final=True)
        y, z = dwc.block_norm_fwd(s @ p.w_out, z, p.gamma_post, p.gamma_pre, None, p.scale, eps=EPS)
        states.append((conv_state, scan_state))
    return y, states


def token(z, params: list, states: list):
    """The output of one more position; the states move on in place.  z: sequences x width."""
    y = first_norm(z, params[0].w_in.dtype)[0]
    for p, (conv_state, scan_state) in zip(params, states):
        inner = p.A.shape[0]
        h = y @ p.w_in
        c = dwc.causal_conv_step(h[:, :inner], conv_state, p.conv, p.conv_bias, "silu")
        dt, B, C = split(c @ p.w_x, p)
        s = dwc.selective_scan_step(c, dt, p.A, B, C, scan_state, p.D, h[:, inner:], p.dt_bias)
        y, z = dwc.block_norm_fwd(s @ p.w_out, z, p.gamma_post, p.gamma_pre, None, p.scale, eps=EPS)
    return y


def generate(z, params: list, tokens: int):
    """Each output is the next position's input: sequences x tokens x width."""
    y, states = prompt(z, params)
    x = y[:, -1].float().contiguous()
    # warm up on another stream and on copies of the states, then capture one token and replay it
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        token(x, params, [(a.clone(), b.clone()) for a, b in states])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token(x, params, states)
    outputs = []
    for _ in range(tokens):
        graph.replay()
        outputs.append(out.to(torch.float32, copy=True))      # (the graph writes the same tensor again)
        x.copy_(out)
    return torch.stack(outputs, 1)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="bf16")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--blocks", type=int, default=3)
    ap.add_argument("--shape", type=int, nargs=3, default=(8, 512, 256), metavar=("B", "T", "W"))
    ap.add_argument("--states", type=int, default=16)
    ap.add_argument("--taps", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=16)
    a = ap.parse_args()
    dtype = torch.float32 if a.dtype == "f32" else torch.bfloat16
    params = make_params(a.blocks, a.shape[-1], 2 * a.shape[-1], a.states, a.taps, dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    z, target = (torch.randn(*a.shape, generator=g, device="cuda") for _ in range(2))
    for step in range(a.steps):
        loss = train_step(z, target, params, rate=0.05 * a.shape[-1])
        if step % 5 == 0 or step == a.steps - 1:
            print(f"step {step:3d}  loss {float(loss):.4f}")
    print("generated", tuple(generate(z, params, a.tokens).shape))


if __name__ == "__main__":
    main()
