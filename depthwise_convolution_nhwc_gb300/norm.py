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

from . import DwcError, load_library

_CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_F32 = torch.float32

# The current stream's handle without building a Stream object (a microsecond of a small call).
_stream_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


@functools.lru_cache(maxsize=None)
def _fn(name: str):
    return getattr(load_library(), name)


def _code(dtype) -> int:
    code = _CODE.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype} (fp32, bf16 or fp16)")
    return code


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
    """(shape, device index, channels, row stride) of a tensor on a CUDA device."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device (no CPU fallback)")
    shape = t.shape
    if not shape or shape[-1] < 1:
        raise ValueError(f"{what} must be [..., C] with at least one channel")
    return shape, dev, shape[-1], shape[-1] if t.is_contiguous() else _stride(t, what)


def _like(t, shape, dev, dtype, what: str) -> int:
    """Row stride of a second tensor of that shape (dtype None: any)."""
    if t.shape != shape or t.get_device() != dev or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{what} must be a {tuple(shape)} {dtype or ''} tensor on cuda:{dev} "
                         f"(got {tuple(t.shape)} {t.dtype} on {t.device})")
    return shape[-1] if t.is_contiguous() else _stride(t, what)


def _out(t, like, dtype, what: str):
    """A dense output of `like`'s shape: the caller's, checked, or a new one."""
    if t is None:
        if like.is_contiguous():
            return torch.empty_like(like, dtype=dtype)
        return torch.empty(like.shape, dtype=dtype, device=like.device)
    if t.shape != like.shape or t.dtype != dtype or t.get_device() != like.get_device() or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {tuple(like.shape)} {dtype} tensor on {like.device} "
                         f"(got {tuple(t.shape)} {t.dtype} on {t.device})")
    return t


def _param(t, C: int, dev: int, what: str) -> int:
    """Pointer of gamma or beta."""
    if t.numel() != C or t.dim() != 1 or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what} must hold {C} values on cuda:{dev} (got {tuple(t.shape)} on {t.device})")
    return t.data_ptr()


def _params(gamma, beta, C: int, dev: int):
    """(gamma's pointer, beta's, their type code)."""
    g = None if gamma is None else _param(gamma, C, dev, "gamma")
    b = None if beta is None else _param(beta, C, dev, "beta")
    if gamma is None:
        return g, b, 0 if beta is None else _code(beta.dtype)
    if beta is not None and beta.dtype != gamma.dtype:
        raise ValueError("gamma and beta must have one dtype")
    return g, b, _code(gamma.dtype)


def _stat(t, lead, dev: int, what: str) -> int:
    if t.shape != lead or t.dtype != _F32 or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {tuple(lead)} fp32 tensor on cuda:{dev} "
                         f"(got {tuple(t.shape)} {t.dtype} on {t.device})")
    return t.data_ptr()


_M64 = 2 ** 64 - 1


def _random(p, seed, offset, dev: int):
    """(p, seed, offset, step pointer) of a dropout."""
    p = float(p)
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must be in [0, 1] (got {p})")
    if isinstance(offset, torch.Tensor):
        if offset.dtype != torch.int64 or offset.numel() != 1 or offset.get_device() != dev:
            raise ValueError("an offset on the device must be one int64 value on the tensors' device")
        return p, int(seed) & _M64, 0, offset.data_ptr()
    return p, int(seed) & _M64, int(offset) & _M64, None


def _run(dev: int, name: str, *args) -> None:
    """The library call on the current stream of device `dev`, with that device current."""
    if dev == torch.cuda.current_device():
        code = _fn(name)(*args, _stream_handle(dev))
    else:
        with torch.cuda.device(dev):
            code = _fn(name)(*args, _stream_handle(dev))
    if code != 0:
        raise DwcError(name, code)


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
    shape, dev, C, ld = _rows(x, "x")
    dtype = x.dtype
    od = out_dtype or (dtype if out is None else out.dtype)
    g, b, pt = _params(gamma, beta, C, dev)
    y = _out(out, x, od, "out")
    if not stats:
        _run(dev, "dwc_layer_norm_fwd", x.data_ptr(), ld, g, b, pt, eps, y.data_ptr(), None, None,
             x.numel() // C, C, _code(dtype), _code(od))
        return y
    mean = torch.empty(shape[:-1], dtype=_F32, device=x.device)
    rstd = torch.empty_like(mean)
    _run(dev, "dwc_layer_norm_fwd", x.data_ptr(), ld, g, b, pt, eps, y.data_ptr(), mean.data_ptr(),
         rstd.data_ptr(), x.numel() // C, C, _code(dtype), _code(od))
    return y, mean, rstd


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(dev: int, rows: int, C: int) -> int:
    with torch.cuda.device(dev):
        return int(_fn("dwc_layer_norm_bwd_workspace_size")(rows, C))


def _param_grads(x, dev: int, rows: int, C: int):
    """(dgamma, dbeta, workspace) of a backward pass.  The workspace comes from PyTorch's allocator
    call by call, so it belongs to the call's stream (or graph) and to no other."""
    dgamma = torch.empty(C, dtype=_F32, device=x.device)
    return dgamma, torch.empty_like(dgamma), torch.empty(_workspace_bytes(dev, rows, C), dtype=torch.uint8,
                                                         device=x.device)


def layer_norm_bwd(dy, x, mean, rstd, gamma=None, out=None, param_grads: bool = True, stream=None):
    """(dx, dgamma, dbeta) of ``layer_norm_fwd`` from dy, its x and its statistics: dx in x's
    dtype, dgamma and dbeta fp32 (None without ``param_grads``)."""
    if stream is not None:
        return _on(stream, layer_norm_bwd, dy, x, mean, rstd, gamma, out, param_grads)
    shape, dev, C, ld = _rows(x, "x")
    rows, dtype, lead = x.numel() // C, x.dtype, shape[:-1]
    lddy = _like(dy, shape, dev, None, "dy")
    g, _, pt = _params(gamma, None, C, dev)
    m, r = _stat(mean, lead, dev, "mean"), _stat(rstd, lead, dev, "rstd")
    dx = _out(out, x, dtype, "out")
    dgamma = dbeta = dg = db = w = None
    n = 0
    if param_grads:
        dgamma, dbeta, ws = _param_grads(x, dev, rows, C)
        dg, db, w, n = dgamma.data_ptr(), dbeta.data_ptr(), ws.data_ptr(), ws.numel()
    _run(dev, "dwc_layer_norm_bwd", dy.data_ptr(), lddy, x.data_ptr(), ld, m, r, g, pt, dx.data_ptr(), dg, db,
         rows, C, _code(dtype), _code(dy.dtype), w, n)
    return dx, dgamma, dbeta


def _dropout(name, x, p, seed, offset, out, what):
    _, dev, C, ld = _rows(x, what)
    p, seed, offset, step = _random(p, seed, offset, dev)
    dtype = x.dtype
    y = _out(out, x, dtype, "out")
    _run(dev, name, x.data_ptr(), ld, y.data_ptr(), x.numel() // C, C, p, seed, offset, step, _code(dtype))
    return y


def dropout_fwd(x, p: float, seed: int, offset=0, out=None, stream=None):
    """x / (1 - q) where kept, 0 where dropped, with probability q = p to the nearest 2^-16;
    ``out`` may be x."""
    if stream is not None:
        return _on(stream, dropout_fwd, x, p, seed, offset, out)
    return _dropout("dwc_dropout_fwd", x, p, seed, offset, out, "x")


def dropout_bwd(dy, p: float, seed: int, offset=0, out=None, stream=None):
    """dx of ``dropout_fwd`` with the same p, seed and offset; ``out`` may be dy."""
    if stream is not None:
        return _on(stream, dropout_bwd, dy, p, seed, offset, out)
    return _dropout("dwc_dropout_bwd", dy, p, seed, offset, out, "dy")


def add_layer_norm_fwd(x, res, gamma=None, beta=None, eps: float = 1e-5, p: float = 0.0, seed: int = 0,
                       offset=0, out=None, z=None, stats: bool = False, stream=None):
    """z = res + dropout(x), y = layer_norm(z) in one pass; (y, z), or (y, z, mean, rstd) with
    ``stats``.  y has x's dtype, z has res's: the same, or fp32 with a 16-bit x.  ``z`` may be
    res (an update of the residual stream in place)."""
    if stream is not None:
        return _on(stream, add_layer_norm_fwd, x, res, gamma, beta, eps, p, seed, offset, out, z, stats)
    shape, dev, C, ldx = _rows(x, "x")
    ldr = _like(res, shape, dev, None, "res")
    p, seed, offset, step = _random(p, seed, offset, dev)
    g, b, pt = _params(gamma, beta, C, dev)
    dtype, rdtype = x.dtype, res.dtype
    y = _out(out, x, dtype, "out")
    z = _out(z, res, rdtype, "z")
    mean = rstd = m = r = None
    if stats:
        mean = torch.empty(shape[:-1], dtype=_F32, device=x.device)
        rstd = torch.empty_like(mean)
        m, r = mean.data_ptr(), rstd.data_ptr()
    _run(dev, "dwc_add_layer_norm_fwd", x.data_ptr(), ldx, res.data_ptr(), ldr, p, seed, offset, step, g, b, pt,
         eps, z.data_ptr(), y.data_ptr(), m, r, x.numel() // C, C, _code(dtype), _code(rdtype))
    return (y, z, mean, rstd) if stats else (y, z)


def add_layer_norm_bwd(dy, z, mean, rstd, gamma=None, dz=None, p: float = 0.0, seed: int = 0, offset=0,
                       param_grads: bool = True, stream=None):
    """(dx, dres, dgamma, dbeta) of ``add_layer_norm_fwd``: dres = dz + layer_norm_bwd(dy) in z's
    dtype, dx = the dropout map of dres in dy's.  ``dz``: the gradient that reaches z from the rest
    of the residual stream (None: zero).  Without dropout and with one dtype dx is dres."""
    if stream is not None:
        return _on(stream, add_layer_norm_bwd, dy, z, mean, rstd, gamma, dz, p, seed, offset, param_grads)
    shape, dev, C, ldz = _rows(z, "z")
    rows, zdtype, lead, dtype = z.numel() // C, z.dtype, shape[:-1], dy.dtype
    lddy = _like(dy, shape, dev, None, "dy")
    lddz = C if dz is None else _like(dz, shape, dev, zdtype, "dz")
    p, seed, offset, step = _random(p, seed, offset, dev)
    g, _, pt = _params(gamma, None, C, dev)
    m, r = _stat(mean, lead, dev, "mean"), _stat(rstd, lead, dev, "rstd")
    dres = _out(None, z, zdtype, "dres")
    dx = dres if p == 0.0 and dtype == zdtype else _out(None, dy, dtype, "dx")
    dgamma = dbeta = dg = db = w = None
    n = 0
    if param_grads:
        dgamma, dbeta, ws = _param_grads(z, dev, rows, C)
        dg, db, w, n = dgamma.data_ptr(), dbeta.data_ptr(), ws.data_ptr(), ws.numel()
    _run(dev, "dwc_add_layer_norm_bwd", dy.data_ptr(), lddy, None if dz is None else dz.data_ptr(), lddz,
         z.data_ptr(), ldz, m, r, g, pt, p, seed, offset, step, None if dx is dres else dx.data_ptr(),
         dres.data_ptr(), dg, db, rows, C, _code(dtype), _code(zdtype), w, n)
    return dx, dres, dgamma, dbeta


__all__ = ["layer_norm_fwd", "layer_norm_bwd", "dropout_fwd", "dropout_bwd", "add_layer_norm_fwd",
           "add_layer_norm_bwd"]
