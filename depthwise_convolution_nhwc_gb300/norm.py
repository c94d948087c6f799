"""Layer norm, dropout, their residual form and the block norm over channels-last rows.

Binding over the C ABI in ``include/dwc_norm.h``.  Tensors are ``[..., C]`` on a CUDA device, fp32,
bf16 or fp16, with adjacent channels and one stride between rows (a slice of a larger tensor's
channels or tokens is taken as it is); outputs are dense.  An output that a call is given (``out``, ``z``) may
be one of its inputs itself, dense and of the output's dtype (an update in place), and must not
overlap them in any other way (ValueError).  Work runs on the current CUDA stream
of the tensors' device, or on ``stream``; outputs and workspaces are then allocated for that
stream and the inputs are recorded on it.  Nothing falls back to the CPU.

    y, mean, rstd = layer_norm_fwd(x, gamma, beta, stats=True)
    dx, dgamma, dbeta = layer_norm_bwd(dy, x, mean, rstd, gamma)

    y = dropout_fwd(x, 0.1, seed, offset);   dx = dropout_bwd(dy, 0.1, seed, offset)

    # z = res + dropout(x), y = layer_norm(z): the end of one residual branch, the norm of the next
    y, z, mean, rstd = add_layer_norm_fwd(x, res, gamma, beta, p=0.1, seed=seed, offset=k, stats=True)
    dx, dres, dgamma, dbeta = add_layer_norm_bwd(dy, z, mean, rstd, gamma, dz, 0.1, seed, k)

    # z = alpha res + scale act(gate) rms_norm(x), y = rms_norm(z): the norms after a block and before the next
    y, z, rstd_post, rstd_pre = block_norm_fwd(x, res, gamma_post, gamma_pre, gate, scale, stats=True)
    dx, dres, dgate, dgamma_post, dgamma_pre, dscale = block_norm_bwd(dy, x, z, rstd_post, rstd_pre, gamma_post,
                                                                      gamma_pre, gate, scale, dz=dz)

The dropout mask is a function of (seed, offset, element index) and is drawn again in the
backward pass.  Use another offset for every dropout of a step and another seed or offset range
for every step; an ``offset`` that is a one-element int64 CUDA tensor is read on the device when
the kernel runs, so a captured CUDA graph draws new masks as the program advances it.
"""
from __future__ import annotations

import torch

from . import DwcError, load_library

_module = None


def _host():
    """The compiled host path (``csrc/dwc_norm_py.cpp``): argument checks, output allocation and the
    library call of each operator as one C++ function.  An error if it was not built."""
    global _module
    if _module is None:
        load_library()
        try:
            from . import _norm_host
        except ImportError as e:
            raise RuntimeError("_norm_host.so is missing or does not fit this PyTorch: build it with "
                               "depthwise_convolution_nhwc_gb300.build()") from e
        _norm_host.set_error(DwcError)
        _module = _norm_host
    return _module


def _stride(t, what: str) -> int:
    """Elements between the rows of [..., C]: one stride over all leading axes, adjacent channels."""
    return _host().row_stride(t, what)


def _on(stream, f, *args):
    """The call f(*args), its allocations included, on `stream`."""
    tensors = [t for t in args if isinstance(t, torch.Tensor) and t.is_cuda]
    for t in tensors:
        if t.device != stream.device:
            raise ValueError(f"stream is on {stream.device}, a tensor on {t.device}")
    with torch.cuda.stream(stream):
        out = f(*args)
    for t in tensors:
        t.record_stream(stream)
    return out


def layer_norm_fwd(x, gamma=None, beta=None, eps: float = 1e-5, out=None, out_dtype=None,
                   stats: bool = False, stream=None):
    """y = (x - mean) * rstd * gamma + beta over the last axis; y, or (y, mean, rstd) with
    ``stats`` (fp32, what the backward pass needs).  y has x's dtype, or ``out_dtype`` (``out``'s):
    a 16-bit type for fp32 x.  gamma and beta: C values of one dtype each, or None."""
    if stream is not None:
        return _on(stream, layer_norm_fwd, x, gamma, beta, eps, out, out_dtype, stats)
    return (_module or _host()).layer_norm_fwd(x, gamma, beta, eps, out, out_dtype, bool(stats))


def layer_norm_bwd(dy, x, mean, rstd, gamma=None, out=None, param_grads: bool = True, stream=None):
    """(dx, dgamma, dbeta) of ``layer_norm_fwd`` from dy, its x and its statistics: dx in x's
    dtype, dgamma and dbeta fp32 (None without ``param_grads``)."""
    if stream is not None:
        return _on(stream, layer_norm_bwd, dy, x, mean, rstd, gamma, out, param_grads)
    return (_module or _host()).layer_norm_bwd(dy, x, mean, rstd, gamma, out, bool(param_grads))


def dropout_fwd(x, p: float, seed: int, offset=0, out=None, stream=None):
    """x / (1 - q) where kept, 0 where dropped, with probability q = p to the nearest 2^-16."""
    if stream is not None:
        return _on(stream, dropout_fwd, x, p, seed, offset, out)
    return (_module or _host()).dropout_fwd(x, p, seed, offset, out)


def dropout_bwd(dy, p: float, seed: int, offset=0, out=None, stream=None):
    """dx of ``dropout_fwd`` with the same p, seed and offset."""
    if stream is not None:
        return _on(stream, dropout_bwd, dy, p, seed, offset, out)
    return (_module or _host()).dropout_bwd(dy, p, seed, offset, out)


def add_layer_norm_fwd(x, res, gamma=None, beta=None, eps: float = 1e-5, p: float = 0.0, seed: int = 0,
                       offset=0, out=None, z=None, stats: bool = False, stream=None):
    """z = res + dropout(x), y = layer_norm(z) in one pass; (y, z), or (y, z, mean, rstd) with
    ``stats``.  y has x's dtype, z has res's: the same, or fp32 with a 16-bit x.  With z=res the
    residual stream is updated in place."""
    if stream is not None:
        return _on(stream, add_layer_norm_fwd, x, res, gamma, beta, eps, p, seed, offset, out, z, stats)
    return (_module or _host()).add_layer_norm_fwd(x, res, gamma, beta, eps, p, seed, offset, out, z, bool(stats))


def add_layer_norm_bwd(dy, z, mean, rstd, gamma=None, dz=None, p: float = 0.0, seed: int = 0, offset=0,
                       param_grads: bool = True, stream=None):
    """(dx, dres, dgamma, dbeta) of ``add_layer_norm_fwd``: dres = dz + layer_norm_bwd(dy) in z's
    dtype, dx = the dropout map of dres in dy's.  ``dz``: the gradient that reaches z from the rest
    of the residual stream (None: zero).  Without dropout and with one dtype dx is dres."""
    if stream is not None:
        return _on(stream, add_layer_norm_bwd, dy, z, mean, rstd, gamma, dz, p, seed, offset, param_grads)
    return (_module or _host()).add_layer_norm_bwd(dy, z, mean, rstd, gamma, dz, p, seed, offset, bool(param_grads))


def block_norm_fwd(x, res, gamma_post=None, gamma_pre=None, gate=None, scale=None, alpha: float = 1.0, act: str = "silu",
                   eps: float = 1e-5, out=None, z=None, stats: bool = False, stream=None):
    """z = alpha * res + scale * act(gate) * rms_norm(x) * gamma_post, y = rms_norm(z) * gamma_pre in one pass:
    the norm behind a block with its gate and scale, the residual sum and the norm in front of the next block.
    (y, z), or (y, z, rstd_post, rstd_pre) with ``stats``.  y and gate have x's dtype, z has res's: the same, or
    fp32 with a 16-bit x.  gamma_post, gamma_pre, scale: C values of one dtype each, or None; act "none",
    "sigmoid" or "silu".  With z=res the residual stream is updated in place."""
    if stream is not None:
        return _on(stream, block_norm_fwd, x, res, gamma_post, gamma_pre, gate, scale, alpha, act, eps, out, z, stats)
    return (_module or _host()).block_norm_fwd(x, res, gamma_post, gamma_pre, gate, scale, alpha, act, eps, out, z,
                                               bool(stats))


def block_norm_bwd(dy, x, z, rstd_post, rstd_pre, gamma_post=None, gamma_pre=None, gate=None, scale=None,
                   alpha: float = 1.0, act: str = "silu", dz=None, param_grads: bool = True, stream=None):
    """(dx, dres, dgate, dgamma_post, dgamma_pre, dscale) of ``block_norm_fwd`` from dy, ``dz`` (the gradient that
    reaches z from the rest of the residual stream; None: zero), its x, z, statistics and parameters: dx and dgate
    in x's dtype, dres in z's, the others fp32 (None for what the call does not have, or without
    ``param_grads``)."""
    if stream is not None:
        return _on(stream, block_norm_bwd, dy, x, z, rstd_post, rstd_pre, gamma_post, gamma_pre, gate, scale, alpha, act,
                   dz, param_grads)
    return (_module or _host()).block_norm_bwd(dy, x, z, rstd_post, rstd_pre, gamma_post, gamma_pre, gate, scale, alpha,
                                               act, dz, bool(param_grads))


__all__ = ["layer_norm_fwd", "layer_norm_bwd", "dropout_fwd", "dropout_bwd", "add_layer_norm_fwd",
           "add_layer_norm_bwd", "block_norm_fwd", "block_norm_bwd"]
