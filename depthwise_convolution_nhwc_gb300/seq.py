"""Operators along sequences, per channel: the short causal depthwise convolution and the selective
scan of state space layers, forward, backward and for single tokens.

Binding over the C ABI in ``include/dwc_seq.h``.  Sequences are a batch ``[B, T, C]``, or packed one
behind the other as ``[rows, C]`` with ``offsets``, the int32 vector (on the device) of their first
rows and the end of the last one; a sequence may be empty, but rows of no sequence (offsets of one
entry) are refused.  Tensors are on a CUDA device, fp32, bf16 or fp16, with adjacent channels and any strides between sequences and positions (slices of a
projection's output are taken as they are); outputs are dense.  Packed rows in front of the first and
behind the last sequence are not read; an ``out`` keeps what it holds there, new outputs are zero.
Work runs on the current CUDA stream of the tensors' device, or on ``stream``.  Nothing falls back to
the CPU.

    y = causal_conv_fwd(x, w, bias, "silu")                       # w: [taps, C]
    dx, dw, dbias, _ = causal_conv_bwd(dy, x, w, bias, "silu")
    y, saved = selective_scan_fwd(u, dt, A, B, C, D, z, dt_bias, save=True)
    du, ddt, dA, dB, dC, dD, dz, ddt_bias, _ = selective_scan_bwd(dy, u, dt, A, B, C, saved, D, z, dt_bias)

A prompt leaves its states with ``final=True``; single tokens then go on from them in place:

    y, conv_state = causal_conv_fwd(x, w, bias, "silu", final=True)          # [B, taps - 1, C]
    y, scan_state = selective_scan_fwd(u, dt, A, B, C, D, z, dt_bias, final=True)   # fp32 [B, C, N]
    y1 = causal_conv_step(x1, conv_state, w, bias, "silu")                     # x1: [B, C]
    y1 = selective_scan_step(u1, dt1, A, B1, C1, scan_state, D, z1, dt_bias)
"""
from __future__ import annotations

from . import norm
from .norm import _host, _on


def causal_conv_fwd(x, w, bias=None, act: str = "none", state=None, offsets=None, out=None, final: bool = False,
                    stream=None):
    """y[t] = act(bias + sum_k w[k] * x[t - taps + 1 + k]) per channel; y, or (y, state) with ``final``.
    act: "none" or "silu".  w: [taps, C], up to 16 taps, and bias: C values, of one dtype.  ``state``: the
    taps - 1 inputs before each sequence's first position, [sequences, taps - 1, C] in x's dtype (None:
    zeros); the one returned holds the last inputs, for a later call."""
    if stream is not None:
        return _on(stream, causal_conv_fwd, x, w, bias, act, state, offsets, out, final)
    return (norm._module or _host()).causal_conv_fwd(x, w, bias, act, state, offsets, out, bool(final))


def causal_conv_bwd(dy, x, w, bias=None, act: str = "none", state=None, offsets=None, dfinal=None,
                    param_grads: bool = True, stream=None):
    """(dx, dw, dbias, dstate) of ``causal_conv_fwd`` from dy and its inputs: dx and dstate in x's dtype
    (dstate None without ``state``), dw and dbias fp32 (None without ``param_grads``; dbias None without
    bias).  ``dfinal``: the gradient of the returned state."""
    if stream is not None:
        return _on(stream, causal_conv_bwd, dy, x, w, bias, act, state, offsets, dfinal, param_grads)
    return (norm._module or _host()).causal_conv_bwd(dy, x, w, bias, act, state, offsets, dfinal, bool(param_grads))


def causal_conv_step(x, state, w, bias=None, act: str = "none", out=None, stream=None):
    """y of one position for each sequence, x [sequences, C]; ``state`` moves on by it in place."""
    if stream is not None:
        return _on(stream, causal_conv_step, x, state, w, bias, act, out)
    return (norm._module or _host()).causal_conv_step(x, state, w, bias, act, out)


def selective_scan_fwd(u, dt, A, B, C, D=None, z=None, dt_bias=None, softplus: bool = True, state=None, offsets=None,
                       out=None, final: bool = False, save: bool = False, stream=None):
    """h_t = exp(delta A) h_{t-1} + delta u B_t, y_t = (C_t . h_t + D u) * silu(z), with delta = softplus(dt +
    dt_bias) (or dt + dt_bias); y, then the last states with ``final``, then with ``save`` what
    ``selective_scan_bwd`` needs.  u, dt, z: positions x channels; A: fp32 [channels, N], N up to 128; B, C:
    positions x N, or positions x groups x N (a group's channels are adjacent), in u's dtype; D, dt_bias:
    fp32, a value per channel.  ``state``: fp32 [sequences, channels, N] (None: zeros)."""
    if stream is not None:
        return _on(stream, selective_scan_fwd, u, dt, A, B, C, D, z, dt_bias, softplus, state, offsets, out, final, save)
    return (norm._module or _host()).selective_scan_fwd(u, dt, A, B, C, D, z, dt_bias, bool(softplus), state, offsets, out,
                                                        bool(final), bool(save))


def selective_scan_bwd(dy, u, dt, A, B, C, saved, D=None, z=None, dt_bias=None, softplus: bool = True, offsets=None,
                       dfinal=None, state_grad: bool = False, stream=None):
    """(du, ddt, dA, dB, dC, dD, dz, ddt_bias, dstate) of ``selective_scan_fwd`` from dy, its inputs and its
    ``saved``: gradients of u, dt, z, B and C in their dtype, the others fp32 (None for an input that is None, and
    dstate without ``state_grad``).  ``dfinal``: the gradient of the last states."""
    if stream is not None:
        return _on(stream, selective_scan_bwd, dy, u, dt, A, B, C, saved, D, z, dt_bias, softplus, offsets, dfinal, state_grad)
    return (norm._module or _host()).selective_scan_bwd(dy, u, dt, A, B, C, saved, D, z, dt_bias, bool(softplus), offsets,
                                                        dfinal, bool(state_grad))


def selective_scan_step(u, dt, A, B, C, state, D=None, z=None, dt_bias=None, softplus: bool = True, out=None, stream=None):
    """y of one position for each sequence, u [sequences, channels]; ``state`` moves on by it in place."""
    if stream is not None:
        return _on(stream, selective_scan_step, u, dt, A, B, C, state, D, z, dt_bias, softplus, out)
    return (norm._module or _host()).selective_scan_step(u, dt, A, B, C, state, D, z, dt_bias, bool(softplus), out)


__all__ = ["causal_conv_fwd", "causal_conv_bwd", "causal_conv_step", "selective_scan_fwd", "selective_scan_bwd",
           "selective_scan_step"]
