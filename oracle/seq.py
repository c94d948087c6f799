"""fp64 definitions of the operators along sequences and of the block norm, with error bounds (numpy;
nothing shared with the CUDA path).  See ``include/dwc_seq.h`` and ``include/dwc_norm.h`` for the operations.

Every quantity is a ``Val``: its fp64 value `v` and `e`, how far an fp32 evaluation may be from it, element by
element.  An operation adds its operands' errors as they reach its result and one rounding, u = 2^-24 of the result; a
fused multiply-add rounds once where two are counted.  A sum of terms that pass through at most D additions
adds D * u * sum|terms|.  ``exp`` (4 u), reciprocals and quotients (3 u) and ``log1p`` (4 u) have the error bounds
that the CUDA programming guide gives for ``expf``, ``__fdividef`` and ``ex2.approx`` (2 ulp, an ulp
being at most 2 u) or that the kernels' own series have, with one u to spare.
"""
from __future__ import annotations

import numpy as np

from .norm import TINY, U

u = U["f32"]
# beside results that fp32 cannot hold relative errors of: exp2 flushes results below 2^-126 to zero, a quotient by
# more than 2^126 (1 + exp(-v) from v = -87.3 on) gives zero, which silu multiplies by v
SMALL = 2.0 ** -118


class Val:
    """A value and the bound of its error in an fp32 evaluation."""
    __array_priority__ = 100.0

    def __init__(self, v, e=0.0):
        self.v = np.asarray(v, np.float64)
        self.e = np.broadcast_to(np.asarray(e, np.float64), self.v.shape)

    def _like(self, v, e, roundings=1.0):
        return Val(v, e + roundings * u * np.abs(v) + SMALL)

    def __add__(self, o):
        o = val(o)
        return self._like(self.v + o.v, self.e + o.e)

    def __sub__(self, o):
        o = val(o)
        return self._like(self.v - o.v, self.e + o.e)

    def __rsub__(self, o):
        return val(o) - self

    def __mul__(self, o):
        o = val(o)
        return self._like(self.v * o.v, np.abs(self.v) * o.e + np.abs(o.v) * self.e + self.e * o.e)

    __radd__, __rmul__ = __add__, __mul__

    def __getitem__(self, k):
        return Val(self.v[k], self.e[k])

    def sum(self, axis, depth=None, keepdims=False):
        """Sum over axes, each term passing through at most `depth` additions."""
        n = np.prod([self.v.shape[a] for a in (axis if isinstance(axis, tuple) else (axis,))])
        d = min(n, depth if depth is not None else n)
        e = self.e.sum(axis, keepdims=keepdims) + d * u * (np.abs(self.v) + self.e).sum(axis, keepdims=keepdims)
        return Val(self.v.sum(axis, keepdims=keepdims), e + SMALL)

    def reshape(self, *shape):
        return Val(self.v.reshape(*shape), self.e.reshape(*shape))

    def rounded(self, t):
        """Bound of the value stored as type t."""
        return 1.01 * (self.e + U[t] * (np.abs(self.v) + self.e)) + TINY[t]


def val(x):
    return x if isinstance(x, Val) else Val(x)


def stack(list_, axis=0):
    return Val(np.stack([x.v for x in list_], axis), np.stack([x.e for x in list_], axis))


def exp(x):
    v = np.exp(x.v)
    # the argument's error, its scaling by log2(e) (two roundings) and the function's
    return Val(v, v * (np.expm1(np.minimum(x.e + 2 * u * np.abs(x.v), 50.0)) + 4 * u) + SMALL)


def sigmoid(x):
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-x.v))
    # 1 / (1 + 2^(-x log2(e))): the exponential's relative error (its argument's, the constant's and the product's
    # roundings, 2 u |x|, and its own, 4 u) counts by its share 1 - s, then a sum and a quotient
    return Val(s, s * (1 - s) * (np.expm1(np.minimum(x.e + 2 * u * np.abs(x.v), 50.0)) + 4 * u) + 4 * u * s + SMALL)


def silu(x):
    s = sigmoid(x)
    return x * s


def silu_slope(x):
    s = sigmoid(x)
    return s + x * s * (1.0 - s)


def softplus(x):
    v = np.maximum(x.v, 0) + np.log1p(np.exp(-np.abs(x.v)))
    s = 1 / (1 + np.exp(-x.v))
    small = np.log1p(np.exp(-np.abs(x.v)))
    # log1p(e) of a relative error of e = 2^(-|x| log2(e)) (4 u + 2 u |x|, as above) is off by at most as much; its series 8 u (a sum, a quotient of 3 u, the
    # odd series: each step's rounding is scaled by s^2 <= 1/9); then the sum with max(x, 0)
    return Val(v, s * x.e + (12 + 2 * np.abs(x.v)) * u * small + u * v + SMALL)


GATES = {"none": (lambda x: x, lambda x: Val(np.ones_like(x.v))), "sigmoid": (sigmoid, lambda x: sigmoid(x) * (1.0 - sigmoid(x))),
         "silu": (silu, silu_slope)}


# ------------------------------------------------------------------------- causal convolution
# One sequence: x [T, C], w [K, C], state [K - 1, C]; sequences are independent but for the parameters' gradients.

def causal_conv(x, w, bias, act, state):
    """y, the last K - 1 inputs."""
    K, T = w.shape[0], x.shape[0]
    line = np.concatenate((state, x))
    pre = val(np.broadcast_to(bias, x.shape))
    for k in range(K):
        pre = pre + val(w[k]) * line[k:k + T]
    return GATES[act][0](pre), line[T:]


def causal_conv_bwd(dy, x, w, bias, act, state, dfinal, depth):
    """dx, dstate, and the terms of dw (list over taps) and dbias along the positions."""
    K, T = w.shape[0], x.shape[0]
    line = np.concatenate((state, x))
    pre = val(np.broadcast_to(bias, x.shape))
    for k in range(K):
        pre = pre + val(w[k]) * line[k:k + T]
    dpre = val(dy) if act == "none" else val(dy) * silu_slope(pre)
    zeros = np.zeros((K - 1, x.shape[1]))
    ahead = Val(np.concatenate((zeros, dpre.v, zeros)), np.concatenate((zeros, dpre.e, zeros)))
    # the line's gradient: position j (state first) takes w[k] dpre[j - k]
    back = val(np.zeros((K - 1 + T, x.shape[1])))
    for k in range(K):
        back = back + val(w[k]) * ahead[K - 1 - k:2 * K - 2 - k + T]
    back = back + np.concatenate((np.zeros((T, x.shape[1])), dfinal))
    dw = [(dpre * line[k:k + T]).sum(0, depth) for k in range(K)]
    return back[K - 1:], back[:K - 1], stack(dw), dpre.sum(0, depth)


# ------------------------------------------------------------------------------ selective scan
# One sequence: u, dt, z [T, C]; A [C, N]; B, C [T, G, N]; state [C, N].

def _spread(b, t, C):
    """[G, N] of position t for every channel."""
    return np.repeat(b[t], C // b.shape[1], axis=0)


def scan(u_, dt, A, B, Cm, D, z, bias, plus, state, history=None):
    """y, the last state; `history` takes per position (a h[t-1], h, delta)."""
    T, C = u_.shape
    N = A.shape[1]
    x = val(dt) + bias
    delta = softplus(x) if plus else x
    h = val(state)
    ys = []
    for t in range(T):
        d = delta[t].reshape(C, 1)
        # (a position's decay and input; carried states keep their error, so it grows along the sequence as in fp32)
        held = exp(d * A) * h
        now = held + d * u_[t][:, None] * _spread(B, t, C)
        if history is not None:
            history.append((held, now, d))
        ys.append((now * _spread(Cm, t, C)).sum(1, N))
        h = now
    y = stack(ys) if ys else Val(np.zeros((0, C)))
    y = y + val(D) * u_
    return (y * silu(val(z)) if z is not None else y), h


def scan_bwd(dy, u_, dt, A, B, Cm, D, z, bias, plus, state, dfinal, depth):
    """Gradients by name; dB and dC per channel block added up (depth: additions along channels and positions)."""
    T, C = u_.shape
    N, G = A.shape[1], B.shape[1]
    history = []
    y, _ = scan(u_, dt, A, B, Cm, D, None, bias, plus, state, history)
    x = val(dt) + bias
    g = val(dy)
    out = {}
    if z is not None:
        out["dz"] = g * y * silu_slope(val(z))
        g = g * silu(val(z))
    carry = val(dfinal)
    du, ddt, dB, dC, dA = [], [], [], [], []
    for t in range(T - 1, -1, -1):
        held, now, d = history[t]
        gt = g[t].reshape(C, 1)
        dh = carry + gt * _spread(Cm, t, C)
        dC.append((gt * now).reshape(G, C // G, N).sum(1, depth))
        dB.append((dh * (d * u_[t][:, None])).reshape(G, C // G, N).sum(1, depth))
        into = (dh * _spread(B, t, C)).sum(1, N)
        part = dh * held
        du.append(into * d.reshape(C) + val(D) * g[t])
        ddt.append(into * u_[t] + (part * A).sum(1, N))
        dA.append(part * d)
        carry = dh * exp(d * A)
    rows = lambda list_, shape: stack(list_[::-1]) if list_ else Val(np.zeros((0,) + shape))  # noqa: E731
    slope = sigmoid(x) if plus else val(np.ones_like(x.v))
    draw = rows(ddt, (C,)) * slope
    out.update(du=rows(du, (C,)), ddt=draw, dB=rows(dB, (G, N)), dC=rows(dC, (G, N)), dA=rows(dA, (C, N)).sum(0, depth),
               dD=(g * u_).sum(0, depth), ddt_bias=draw.sum(0, depth), dstate=carry)
    return out


# -------------------------------------------------------------------------------- block norm

def _rstd(x, eps, depth):
    C = x.v.shape[1]
    m = (x * x).sum(1, depth) * (1 / C) + eps
    with np.errstate(divide="ignore"):
        v = 1 / np.sqrt(m.v)
        return Val(v, v * (0.5 * m.e / m.v + 4 * u))


def block_norm(x, res, gpost, gpre, gate, scale, alpha, act, eps):
    """y, z, rstd_post, rstd_pre of rows x C arrays."""
    depth = x.shape[1] / 256 + 80
    post = _rstd(val(x), eps, depth)
    m = val(x) * post.reshape(-1, 1) * gpost
    if gate is not None:
        m = m * GATES[act][0](val(gate))
    z = val(res) * alpha + m * scale
    pre = _rstd(z, eps, depth)
    return z * pre.reshape(-1, 1) * gpre, z, post, pre


def block_norm_bwd(dy, x, z, post, pre, gpost, gpre, gate, scale, alpha, act, dz):
    """Gradients by name, from the given statistics."""
    C, rows = x.shape[1], x.shape[0]
    depth, down = C / 256 + 80, rows / 64 + 400
    post, pre = val(post.reshape(-1, 1)), val(pre.reshape(-1, 1))
    zhat, a = val(z) * pre, val(dy) * gpre
    g = pre * (a - zhat * ((a * zhat).sum(1, depth, True) * (1 / C))) + dz
    xhat = val(x) * post
    n = xhat * gpost
    f, slope = GATES[act]
    open_ = f(val(gate)) if gate is not None else val(np.ones_like(x))
    dm = g * scale
    dn = dm * open_
    b = dn * gpost
    out = {"dx": post * (b - xhat * ((b * xhat).sum(1, depth, True) * (1 / C))), "dres": g * alpha,
           "dgamma_post": (dn * xhat).sum(0, down), "dgamma_pre": (val(dy) * zhat).sum(0, down),
           "dscale": (g * open_ * n).sum(0, down)}
    if gate is not None:
        out["dgate"] = dm * n * slope(val(gate))
    return out
