"""Layer norm, dropout and their residual form over channels-last rows.

Binding over the C ABI in ``include/dwc_norm.h``.  Tensors are ``[..., C]`` on a CUDA device, fp32,
bf16 or fp16, with adjacent channels and one stride between rows (a slice of a larger tensor's
channels or tokens is taken as it is); outputs are dense.  Work runs on the current CUDA stream
of the tensors' device, or on ``stream``; outputs and workspaces are then allocated for that
stream and the inputs are recorded on it.  Nothing falls back to the CPU.

    y, mean, rstd = layer_norm_fwd(x, gamma, beta, stats=True)
    dx, dgamma, dbeta = layer_norm_bwd(dy, x, mean, rstd, gamma)

    y = dropout_fwd(x, 0.1, seed, offset);   dx = dropout_bwd(dy, 0.1, seed, offset)

    # z = res + dropout(x), y = layer_norm(z): the end of one residual branch, the norm of the next
    y, z, mean, rstd = add_layer_norm_fwd(x, res, gamma, beta, p=0.1, seed=seed, offset=k, stats=True)
    dx, dres, dgamma, dbeta = add_layer_norm_bwd(dy, z, mean, rstd, gamma, dz, 0.1, seed, k)

The dropout mask is a function of (seed, offset, element index) and is drawn again in the
backward pass.  Use another offset for every dropout of a step and another seed or offset range
for every step; an ``offset`` that is a one-element int64 CUDA tensor is read on the device when
the kernel runs, so a captured CUDA graph draws new masks as the program advances it.
"""
from __future__ import annotations

import functools

import torch

from . import _call, load_library

_CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _code(dtype) -> int:
    try:
        return _CODE[dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {dtype} (fp32, bf16 or fp16)") from None


def _stride(t, what: str) -> int:
    """Elements between the rows of [..., C]: one stride over all leading axes, adjacent channels."""
    C = t.shape[-1]
    if t.is_contiguous():
        return C
    ld, span = None, None
    if C > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what}: channels must be adjacent (stride {t.stride(-1)})")
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if ld is None:
            if s < C:
                raise ValueError(f"{what}: rows overlap (stride {s} between rows of {C})")
            ld, span = s, n * s
        elif s != span:
            raise ValueError(f"{what}: rows must have one stride (got {tuple(t.stride())} for {tuple(t.shape)})")
        else:
            span *= n
    return C if ld is None else ld


def _rows(t, what: str):
    """(rows, C, row stride) of a tensor on a CUDA device."""
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device (no CPU fallback)")
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError(f"{what} must be [..., C] with at least one channel")
    C = t.shape[-1]
    return t.numel() // C, C, _stride(t, what)


def _like(t, x, dtype, what: str) -> int:
    """Row stride of a second tensor of x's shape."""
    if t.shape != x.shape or t.dtype != dtype or t.device != x.device:
        raise ValueError(f"{what} must be a {tuple(x.shape)} {dtype} tensor on {x.device} "
                         f"(got {tuple(t.shape)} {t.dtype} on {t.device})")
    return _stride(t, what)


def _out(t, shape, dtype, x, what: str):
    """A dense output: the caller's, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=x.device)
    if t.shape != shape or t.dtype != dtype or t.device != x.device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {tuple(shape)} {dtype} tensor on {x.device} "
                         f"(got {tuple(t.shape)} {t.dtype} on {t.device})")
    return t


def _param(t, C: int, x, what: str):
    """(pointer, type code) of gamma or beta."""
    if t is None:
        return None, None
    if t.dim() != 1 or t.shape[0] != C or t.device != x.device or not t.is_contiguous():
        raise ValueError(f"{what} must hold {C} values on {x.device} (got {tuple(t.shape)} on {t.device})")
    return t.data_ptr(), _code(t.dtype)


def _params(gamma, beta, C: int, x):
    g, gt = _param(gamma, C, x, "gamma")
    b, bt = _param(beta, C, x, "beta")
    if gt is not None and bt is not None and gt != bt:
        raise ValueError("gamma and beta must have one dtype")
    return g, b, gt if gt is not None else (bt or 0)


def _stat(t, x, what: str) -> int:
    if t.shape != x.shape[:-1] or t.dtype != torch.float32 or t.device != x.device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {tuple(x.shape[:-1])} fp32 tensor on {x.device} "
                         f"(got {tuple(t.shape)} {t.dtype} on {t.device})")
    return t.data_ptr()


def _random(p, seed, offset, x):
    """(p, seed, offset, step pointer) of a dropout."""
    p = float(p)
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must be in [0, 1] (got {p})")
    if isinstance(offset, torch.Tensor):
        if offset.dtype != torch.int64 or offset.numel() != 1 or offset.device != x.device:
            raise ValueError("an offset on the device must be one int64 value on the tensors' device")
        return p, int(seed) & (2 ** 64 - 1), 0, offset.data_ptr()
    return p, int(seed) & (2 ** 64 - 1), int(offset) & (2 ** 64 - 1), None


def _run(x, fn: str, *args) -> None:
    """The library call on the current stream of x's device, with that device current."""
    dev = x.get_device()
    if dev == torch.cuda.current_device():
        _call(fn, *args, torch.cuda.current_stream(dev).cuda_stream)
    else:
        with torch.cuda.device(dev):
            _call(fn, *args, torch.cuda.current_stream(dev).cuda_stream)


def _on_stream(f):
    """``stream``: run the call, its allocations included, on that stream."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        tensors = [t for t in (*args, *kw.values()) if isinstance(t, torch.Tensor)]
        for t in tensors:
            if t.is_cuda and t.device != stream.device:
                raise ValueError(f"stream is on {stream.device}, a tensor on {t.device}")
        with torch.cuda.stream(stream):
            out = f(*args, **kw)
        for t in tensors:
            if t.is_cuda:
                t.record_stream(stream)
        return out
    return call


@_on_stream
def layer_norm_fwd(x, gamma=None, beta=None, eps: float = 1e-5, out=None, out_dtype=None,
                   stats: bool = False):
    """y = (x - mean) * rstd * gamma + beta over the last axis; y, or (y, mean, rstd) with
    ``stats`` (fp32, what the backward pass needs).  y has x's dtype, or ``out_dtype`` (``out``'s):
    a 16-bit type for fp32 x.  gamma and beta: C values of one dtype each, or None."""
    rows, C, ld = _rows(x, "x")
    od = out_dtype or (x.dtype if out is None else out.dtype)
    g, b, pt = _params(gamma, beta, C, x)
    y = _out(out, x.shape, od, x, "out")
    mean = rstd = None
    if stats:
        mean, rstd = (torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device) for _ in range(2))
    _run(x, "dwc_layer_norm_fwd", x.data_ptr(), ld, g, b, pt, eps, y.data_ptr(),
         mean.data_ptr() if stats else None, rstd.data_ptr() if stats else None, rows, C,
         _code(x.dtype), _code(od))
    return (y, mean, rstd) if stats else y


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(device: int, rows: int, C: int) -> int:
    with torch.cuda.device(device):
        return int(load_library().dwc_layer_norm_bwd_workspace_size(rows, C))


def _param_grads(x, rows: int, C: int, wanted: bool):
    """(dgamma, dbeta, workspace) of a backward pass."""
    if not wanted:
        return None, None, None
    grads = torch.empty((2, C), dtype=torch.float32, device=x.device)
    ws = torch.empty(_workspace_bytes(x.get_device(), rows, C), dtype=torch.uint8, device=x.device)
    return grads[0], grads[1], ws


def _ptr(t):
    return None if t is None else t.data_ptr()


@_on_stream
def layer_norm_bwd(dy, x, mean, rstd, gamma=None, out=None, param_grads: bool = True):
    """(dx, dgamma, dbeta) of ``layer_norm_fwd`` from dy, its x and its statistics: dx in x's
    dtype, dgamma and dbeta fp32 (None without ``param_grads``)."""
    rows, C, ld = _rows(x, "x")
    lddy = _like(dy, x, dy.dtype, "dy")
    g, _, pt = _params(gamma, None, C, x)
    m, r = _stat(mean, x, "mean"), _stat(rstd, x, "rstd")
    dx = _out(out, x.shape, x.dtype, x, "out")
    dgamma, dbeta, ws = _param_grads(x, rows, C, param_grads)
    _run(x, "dwc_layer_norm_bwd", dy.data_ptr(), lddy, x.data_ptr(), ld, m, r, g, pt, dx.data_ptr(),
         _ptr(dgamma), _ptr(dbeta), rows, C, _code(x.dtype), _code(dy.dtype), _ptr(ws),
         0 if ws is None else ws.numel())
    return dx, dgamma, dbeta


def _dropout(fn, x, p, seed, offset, out, what):
    rows, C, ld = _rows(x, what)
    p, seed, offset, step = _random(p, seed, offset, x)
    y = _out(out, x.shape, x.dtype, x, "out")
    _run(x, fn, x.data_ptr(), ld, y.data_ptr(), rows, C, p, seed, offset, step, _code(x.dtype))
    return y


@_on_stream
def dropout_fwd(x, p: float, seed: int, offset=0, out=None):
    """x / (1 - q) where kept, 0 where dropped, with probability q = p to the nearest 2^-16;
    ``out`` may be x."""
    return _dropout("dwc_dropout_fwd", x, p, seed, offset, out, "x")


@_on_stream
def dropout_bwd(dy, p: float, seed: int, offset=0, out=None):
    """dx of ``dropout_fwd`` with the same p, seed and offset; ``out`` may be dy."""
    return _dropout("dwc_dropout_bwd", dy, p, seed, offset, out, "dy")


@_on_stream
def add_layer_norm_fwd(x, res, gamma=None, beta=None, eps: float = 1e-5, p: float = 0.0, seed: int = 0,
                       offset=0, out=None, z=None, stats: bool = False):
    """z = res + dropout(x), y = layer_norm(z) in one pass; (y, z), or (y, z, mean, rstd) with
    ``stats``.  y has x's dtype, z has res's: the same, or fp32 with a 16-bit x.  ``z`` may be
    res (an update of the residual stream in place)."""
    rows, C, ldx = _rows(x, "x")
    ldr = _like(res, x, res.dtype, "res")
    p, seed, offset, step = _random(p, seed, offset, x)
    g, b, pt = _params(gamma, beta, C, x)
    y = _out(out, x.shape, x.dtype, x, "out")
    z = _out(z, x.shape, res.dtype, x, "z")
    mean = rstd = None
    if stats:
        mean, rstd = (torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device) for _ in range(2))
    _run(x, "dwc_add_layer_norm_fwd", x.data_ptr(), ldx, res.data_ptr(), ldr, p, seed, offset, step, g, b, pt,
         eps, z.data_ptr(), y.data_ptr(), mean.data_ptr() if stats else None,
         rstd.data_ptr() if stats else None, rows, C, _code(x.dtype), _code(res.dtype))
    return (y, z, mean, rstd) if stats else (y, z)


@_on_stream
def add_layer_norm_bwd(dy, z, mean, rstd, gamma=None, dz=None, p: float = 0.0, seed: int = 0, offset=0,
                       param_grads: bool = True):
    """(dx, dres, dgamma, dbeta) of ``add_layer_norm_fwd``: dres = dz + layer_norm_bwd(dy) in z's
    dtype, dx = the dropout map of dres in dy's.  ``dz``: the gradient that reaches z from the rest
    of the residual stream (None: zero).  Without dropout and with one dtype dx is dres."""
    rows, C, ldz = _rows(z, "z")
    lddy = _like(dy, z, dy.dtype, "dy")
    lddz = C if dz is None else _like(dz, z, z.dtype, "dz")
    p, seed, offset, step = _random(p, seed, offset, z)
    g, _, pt = _params(gamma, None, C, z)
    m, r = _stat(mean, z, "mean"), _stat(rstd, z, "rstd")
    dres = torch.empty(z.shape, dtype=z.dtype, device=z.device)
    dx = dres
    if p != 0.0 or dy.dtype != z.dtype:
        dx = torch.empty(z.shape, dtype=dy.dtype, device=z.device)
    dgamma, dbeta, ws = _param_grads(z, rows, C, param_grads)
    _run(z, "dwc_add_layer_norm_bwd", dy.data_ptr(), lddy, _ptr(dz), lddz, z.data_ptr(), ldz, m, r, g, pt, p,
         seed, offset, step, None if dx is dres else dx.data_ptr(), dres.data_ptr(), _ptr(dgamma), _ptr(dbeta),
         rows, C, _code(dy.dtype), _code(z.dtype), _ptr(ws), 0 if ws is None else ws.numel())
    return dx, dres, dgamma, dbeta


__all__ = ["layer_norm_fwd", "layer_norm_bwd", "dropout_fwd", "dropout_bwd", "add_layer_norm_fwd",
           "add_layer_norm_bwd"]
