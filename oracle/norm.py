"""fp64 definitions of layer norm, dropout and their residual form (numpy; nothing shared with the
CUDA path).  Rows x C arrays in, rows x C arrays out; see ``include/dwc_norm.h`` for the
operations.  ``*_bound`` gives, element by element, how far an fp32 evaluation that rounds its
result once to the output type may be from the definition.

The bounds follow from u = 2^-24 (fp32) and the output type's u_out: a sum of n terms in which no
partial sum is deeper than D additions is off by at most D * u * sum|terms| (first order).  The
kernels add at most C / 256 + 80 terms one after another along a row (threads of a CTA, then
lanes, then warps) and at most rows / 64 + 400 down a column (the rows of one CTA, its row
groups, then the partial sums); each further operation adds one u of its result.  Beyond 10240
channels a cluster of up to 8 CTAs takes the place of a CTA, of which at least 8 run together: a thread
adds at most rows / 8 terms and the partial sums 76, which is within rows / 64 + 400 up to 2900 rows.
"""
from __future__ import annotations

import numpy as np

# unit roundoff 2^-p of p significant bits: the largest relative error of one rounding to nearest
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
# half the distance of the smallest fp16 subnormals (bf16 and fp32 ones are out of sight here)
TINY = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}


def philox4x32_10(counter, key):
    """The 4 words of one block (Salmon et al. 2011, "Parallel random numbers: as easy as 1, 2,
    3"): 4 counter words and 2 key words, low first, as Python integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p0, p1 = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & 0xFFFFFFFF, (p0 >> 32) ^ c[3] ^ k[1], p0 & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def kept(first: int, count: int, p: float, seed: int, offset: int) -> np.ndarray:
    """Which of the elements first .. first + count - 1 are kept."""
    q = int(np.floor(p * 65536 + 0.5))
    g = np.arange(first // 8, (first + count + 7) // 8, dtype=np.uint64)
    lo, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    c = [g & lo, g >> sh, np.full_like(g, offset & 0xFFFFFFFF), np.full_like(g, (offset >> 32) & 0xFFFFFFFF)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        p0, p1 = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(p1 >> sh) ^ c[1] ^ np.uint64(k[0]), p1 & lo, (p0 >> sh) ^ c[3] ^ np.uint64(k[1]), p0 & lo]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    h = np.stack([v for w in c for v in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 1).reshape(-1)
    at = first - first // 8 * 8
    return h[at:at + count] >= np.uint64(q)


def dropout(x, p: float, seed: int, offset: int, first: int = 0):
    q = np.floor(p * 65536 + 0.5) / 65536
    if q == 0:
        return x.copy()
    keep = kept(first, x.size, p, seed, offset).reshape(x.shape)
    with np.errstate(all="ignore"):
        return np.where(keep, x / (1 - q) if q < 1 else 0.0, 0.0)


def layer_norm(x, gamma, beta, eps):
    """y, mean, rstd."""
    mean = x.mean(1)
    with np.errstate(all="ignore"):
        rstd = 1 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
        return (x - mean[:, None]) * rstd[:, None] * gamma + beta, mean, rstd


def layer_norm_bwd(dy, x, mean, rstd, gamma):
    """dx, dgamma, dbeta."""
    xhat = (x - mean[:, None]) * rstd[:, None]
    a = dy * gamma
    dx = rstd[:, None] * (a - a.mean(1, keepdims=True) - xhat * (a * xhat).mean(1, keepdims=True))
    return dx, (dy * xhat).sum(0), dy.sum(0)


def _depth(C: int) -> float:
    return C / 256 + 80


def layer_norm_bound(x, gamma, beta, eps, out: str, e_x=0.0):
    """Bounds of (y, mean, rstd); e_x: how far each element of x is off already (a sum that was
    rounded on the way)."""
    u, D = U["f32"], _depth(x.shape[1])
    e_x = np.broadcast_to(e_x, x.shape)
    y, mean, rstd = layer_norm(x, gamma, beta, eps)
    r = rstd[:, None]
    xhat = np.abs(x - mean[:, None]) * r
    e_mean = (D + 4) * u * np.abs(x).mean(1) + e_x.mean(1)
    # a shift of all differences by e moves the variance by e^2; a rounding of each by its share
    e_rel = 0.5 * ((D + 10) * u + (e_mean * rstd) ** 2) + (xhat * (e_x + 2 * u * np.abs(x)) * r).mean(1) + 4 * u
    e_hat = r * (e_mean[:, None] + 2 * u * np.abs(x) + e_x) + xhat * (e_rel[:, None] + 3 * u)
    e_y = np.abs(gamma) * e_hat + 3 * u * (np.abs(gamma) * xhat + np.abs(beta))
    return 1.01 * (e_y + U[out] * np.abs(y)) + TINY[out], e_mean, e_rel * rstd


def layer_norm_bwd_bound(dy, x, mean, rstd, gamma, out: str, dz=None):
    """Bounds of (dx [+ dz], dgamma, dbeta)."""
    u, D, rows = U["f32"], _depth(x.shape[1]), x.shape[0]
    r = rstd[:, None]
    xhat, a = np.abs(x - mean[:, None]) * r, np.abs(dy * gamma)
    m1, m2 = a.mean(1, keepdims=True), (a * xhat).mean(1, keepdims=True)
    e = r * (4 * u * a + (D + 6) * u * m1 + xhat * (D + 12) * u * m2)
    dx, _, _ = layer_norm_bwd(dy, x, mean, rstd, gamma)
    g = dx
    if dz is not None:
        g = dx + dz
        e = e + u * (np.abs(dx) + np.abs(g))
    Dr = rows / 64 + 400
    e = e + U[out] * np.abs(g) * 1.01 + TINY[out]
    return e, (Dr + 6) * u * (np.abs(dy) * xhat).sum(0), (Dr + 1) * u * np.abs(dy).sum(0)
