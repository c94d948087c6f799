"""Sequence operators and block norm without a GPU: the 64-bit definitions (gradients against differences, parts of
a sequence against the whole) and the refusals of the C ABI and the binding."""
import ctypes
import os

import numpy as np
import pytest
import torch

import depthwise_convolution_nhwc_gb300 as dwc
from oracle import seq as ref

FAKE = 0x10000  # never dereferenced: every case below fails validation first


def differences(loss, args, h=1e-5):
    """Central differences of a scalar function by every element of its arrays."""
    out = []
    for k, a in enumerate(args):
        g = np.empty_like(a)
        for i in np.ndindex(a.shape):
            side = []
            for s in (h, -h):
                moved = [x.copy() for x in args]
                moved[k][i] += s
                side.append(loss(*moved))
            g[i] = (side[0] - side[1]) / (2 * h)
        out.append(g)
    return out


def close(got, want):
    # truncation h^2 and rounding 1e-16 / h are both near 1e-10 at h = 1e-5 for values and derivatives of order 1 to 10
    np.testing.assert_allclose(got, want, rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("T", [1, 2, 7])
def test_causal_conv_gradients(T, act):
    rng = np.random.default_rng(T)
    K, C = 4, 3
    x, w, bias, state, dy, dlast = (rng.standard_normal(s) for s in ((T, C), (K, C), C, (K - 1, C), (T, C), (K - 1, C)))

    def loss(x, w, bias, state):
        y, last = ref.causal_conv(x, w, bias, act, state)
        return (y.v * dy).sum() + (last * dlast).sum()

    dx, dstate, dw, db = ref.causal_conv_bwd(dy, x, w, bias, act, state, dlast, 1)
    for got, want in zip((dx.v, dw.v, db.v, dstate.v), differences(loss, [x, w, bias, state])):
        close(got, want)


@pytest.mark.parametrize("gate,plus", [(True, True), (False, True), (True, False)])
def test_scan_gradients(gate, plus):
    rng = np.random.default_rng(5)
    T, C, N, G = 5, 4, 3, 2
    u, dt, z, dy = (rng.standard_normal((T, C)) for _ in range(4))
    if not plus:
        dt = np.abs(dt) + 0.1
    A = -np.exp(rng.standard_normal((C, N)) * 0.3)
    B, Cm = (rng.standard_normal((T, G, N)) for _ in range(2))
    D, bias = rng.standard_normal(C), 0.3 * rng.standard_normal(C) if plus else np.zeros(C)
    state, dlast = (rng.standard_normal((C, N)) for _ in range(2))

    def loss(u, dt, A, B, Cm, D, z, bias, state):
        y, last = ref.scan(u, dt, A, B, Cm, D, z if gate else None, bias, plus, state)
        return (y.v * dy).sum() + (last.v * dlast).sum()

    got = ref.scan_bwd(dy, u, dt, A, B, Cm, D, z if gate else None, bias, plus, state, dlast, 1)
    want = differences(loss, [u, dt, A, B, Cm, D, z, bias, state])
    for name, w in zip(("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dstate"), want):
        if name == "dz" and not gate:
            continue
        close(got[name].v, w)


def test_parts_of_a_sequence_are_the_whole():
    rng = np.random.default_rng(6)
    T, C, N, K = 9, 2, 3, 4
    x, dt, B, Cm = rng.standard_normal((T, C)), rng.standard_normal((T, C)), *(rng.standard_normal((T, 1, N)) for _ in range(2))
    A, w = -np.exp(rng.standard_normal((C, N))), rng.standard_normal((K, C))
    zero = np.zeros(C)
    whole, last = ref.scan(x, dt, A, B, Cm, zero, None, zero, True, np.zeros((C, N)))
    a, h = ref.scan(x[:4], dt[:4], A, B[:4], Cm[:4], zero, None, zero, True, np.zeros((C, N)))
    b, h = ref.scan(x[4:], dt[4:], A, B[4:], Cm[4:], zero, None, zero, True, h.v)
    np.testing.assert_allclose(np.concatenate((a.v, b.v)), whole.v, rtol=1e-12)
    np.testing.assert_allclose(h.v, last.v, rtol=1e-12)
    for cut in (1, 2, 5):
        whole, last = ref.causal_conv(x, w, zero, "silu", np.zeros((K - 1, C)))
        a, s = ref.causal_conv(x[:cut], w, zero, "silu", np.zeros((K - 1, C)))
        b, s = ref.causal_conv(x[cut:], w, zero, "silu", s)
        np.testing.assert_array_equal(np.concatenate((a.v, b.v)), whole.v)
        np.testing.assert_array_equal(s, last)


@pytest.mark.parametrize("act", ["none", "sigmoid", "silu"])
def test_block_norm_gradients(act):
    rng = np.random.default_rng(7)
    R, C, alpha, eps = 3, 5, 0.8, 1e-3
    x, res, gate, dy, dz = (rng.standard_normal((R, C)) for _ in range(5))
    gpost, gpre, scale = (1 + 0.3 * rng.standard_normal(C) for _ in range(3))

    def loss(x, res, gate, gpost, gpre, scale):
        y, z, _, _ = ref.block_norm(x, res, gpost, gpre, gate, scale, alpha, act, eps)
        return (y.v * dy).sum() + (z.v * dz).sum()

    _, z, post, pre = ref.block_norm(x, res, gpost, gpre, gate, scale, alpha, act, eps)
    got = ref.block_norm_bwd(dy, x, z.v, post.v, pre.v, gpost, gpre, gate, scale, alpha, act, dz)
    names = ("dx", "dres", "dgate", "dgamma_post", "dgamma_pre", "dscale")
    for name, want in zip(names, differences(loss, [x, res, gate, gpost, gpre, scale])):
        close(got[name].v, want)


def test_bounds_hold_for_fp32_arithmetic():
    """The bounds against the same formulas in numpy's fp32 (one rounding an operation)."""
    rng = np.random.default_rng(8)
    f = np.float32
    a, b = rng.standard_normal(1000), rng.standard_normal(1000)
    for exact, got in ((ref.val(a) * b + a, (f(a) * f(b)).astype(f) + f(a)), (ref.silu(ref.val(a) * 9), None),
                       (ref.softplus(ref.val(a) * 9), None)):
        if got is None:
            x = f(a) * f(9)
            want = x / (1 + np.exp(-x)) if exact.v.min() < 0 else np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))
            got = want.astype(f)
        # (the arguments' own rounding to fp32 is not an operation's: allow it apart)
        slack = 4 * ref.u * (np.abs(a) * 9 + np.abs(b) + np.abs(exact.v)) * 2
        assert np.all(np.abs(got - exact.v) <= exact.e + slack)


# ------------------------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dwc.LIB_PATH):
        dwc.build()
    return dwc.load_library()


def conv(count=2, length=5, offsets=None, C=8, K=4, act=2, dtype=0, param=0, x=FAKE, seq=40, row=8, w=FAKE, bias=FAKE,
         state=FAKE):
    return dwc.CausalConv(dwc.Seqs(count, length, offsets), C, K, act, dtype, param, dwc.Rows(x, seq, row), w, bias, state)


def conv_codes(lib, c, y=FAKE, final=FAKE, dy=None, dx=FAKE, ws=FAKE, nws=1 << 30, backward=True):
    codes = {lib.dwc_causal_conv_fwd(c, y, final, None)}
    if backward:
        codes.add(lib.dwc_causal_conv_bwd(c, dy or dwc.Rows(FAKE, 40, 8), None, dx, None, FAKE, FAKE, ws, nws, None))
    assert len(codes) == 1, codes
    return codes.pop()


def scan(count=2, length=5, offsets=None, C=8, N=4, G=2, plus=1, dtype=0, u=FAKE, dt=FAKE, z=FAKE, b=FAKE, c=FAKE, seq=40, row=8,
         A=FAKE, D=FAKE, bias=FAKE):
    v = lambda p: dwc.Rows(p, seq, row)  # noqa: E731
    return dwc.Scan(dwc.Seqs(count, length, offsets), C, N, G, plus, dtype, v(u), v(dt), v(z), v(b), v(c), A, D, bias)


def scan_codes(lib, s, y=FAKE, state=FAKE, saved=FAKE, dy=None, ws=FAKE, nws=1 << 40):
    codes = {lib.dwc_selective_scan_fwd(s, state, y, FAKE, saved, ws, nws, None),
             lib.dwc_selective_scan_bwd(s, dy or dwc.Rows(FAKE, 40, 8), saved, None, y, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                                        FAKE, ws, nws, None)}
    assert len(codes) == 1, codes
    return codes.pop()


INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4


@pytest.mark.parametrize("kw,code", [
    (dict(count=-1), INVALID), (dict(length=-1), INVALID), (dict(C=0), INVALID), (dict(K=0), INVALID), (dict(act=1), INVALID),
    (dict(act=3), INVALID), (dict(dtype=5), INVALID), (dict(param=5), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(row=-1), INVALID), (dict(seq=-1), INVALID), (dict(count=0, length=3, offsets=FAKE), INVALID),
    (dict(K=17), UNSUPPORTED), (dict(C=(1 << 20) + 1), UNSUPPORTED), (dict(count=1 << 16, length=1 << 16), UNSUPPORTED),
    (dict(offsets=FAKE, length=1 << 31), UNSUPPORTED), (dict(C=1 << 20, length=1 << 24), UNSUPPORTED),
    (dict(row=1 << 40), UNSUPPORTED), (dict(x=FAKE + 2), ALIGNMENT), (dict(offsets=FAKE + 2), ALIGNMENT),
    (dict(w=FAKE + 2), ALIGNMENT), (dict(bias=FAKE + 1, param=1), ALIGNMENT), (dict(state=FAKE + 2), ALIGNMENT),
    (dict(dtype=1, x=FAKE + 1), ALIGNMENT)])
def test_causal_conv_refusals(lib, kw, code):
    assert conv_codes(lib, conv(**kw)) == code


def test_causal_conv_outputs_and_workspace(lib):
    c = conv()
    assert lib.dwc_causal_conv_fwd(None, FAKE, None, None) == INVALID
    assert lib.dwc_causal_conv_fwd(c, None, None, None) == INVALID
    assert lib.dwc_causal_conv_fwd(c, FAKE + 2, None, None) == ALIGNMENT
    assert lib.dwc_causal_conv_fwd(c, FAKE, FAKE + 2, None) == ALIGNMENT
    dy = dwc.Rows(FAKE, 40, 8)
    need = lib.dwc_causal_conv_bwd_workspace_size(c)
    assert need >= 5 * 8 * 4 and lib.dwc_causal_conv_bwd_workspace_size(conv(K=17)) == 0
    bwd = lambda dy=dy, dx=FAKE, dw=FAKE, ws=FAKE, n=need: lib.dwc_causal_conv_bwd(  # noqa: E731
        c, dy, None, dx, None, dw, FAKE, ws, n, None)
    assert bwd(dy=None) == INVALID and bwd(dx=None) == INVALID and bwd(dy=dwc.Rows(None, 40, 8)) == INVALID
    assert bwd(dw=FAKE + 2) == ALIGNMENT and bwd(ws=FAKE + 8) == ALIGNMENT
    assert bwd(ws=None) == WORKSPACE and bwd(n=need - 1) == WORKSPACE
    # nothing to do
    assert lib.dwc_causal_conv_fwd(conv(count=0), None, None, None) == 0
    assert lib.dwc_causal_conv_fwd(conv(length=0, x=None), None, None, None) == 0


def test_causal_conv_step_refusals(lib):
    step = lambda c, state=FAKE, stride=24, y=FAKE: lib.dwc_causal_conv_step(c, state, stride, y, None)  # noqa: E731
    assert step(conv()) == INVALID                                     # more than one position
    assert step(conv(length=1, offsets=FAKE)) == INVALID
    one = conv(length=1)
    assert step(one, stride=23) == INVALID and step(one, state=None) == INVALID and step(one, y=None) == INVALID
    assert step(one, state=FAKE + 2) == ALIGNMENT and step(one, stride=1 << 40) == UNSUPPORTED
    assert step(conv(count=0, length=1), state=None, y=None) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(count=-1), INVALID), (dict(length=-1), INVALID), (dict(C=0), INVALID), (dict(N=0), INVALID), (dict(G=0), INVALID),
    (dict(G=3), INVALID), (dict(dtype=3), INVALID), (dict(u=None), INVALID), (dict(dt=None), INVALID), (dict(b=None), INVALID),
    (dict(c=None), INVALID), (dict(A=None), INVALID), (dict(row=-8), INVALID), (dict(N=129), UNSUPPORTED),
    (dict(C=(1 << 20) + 2), UNSUPPORTED), (dict(count=1 << 16, length=1 << 16), UNSUPPORTED), (dict(seq=1 << 41), UNSUPPORTED),
    (dict(u=FAKE + 2), ALIGNMENT), (dict(z=FAKE + 1, dtype=1), ALIGNMENT), (dict(b=FAKE + 1, dtype=2), ALIGNMENT),
    (dict(A=FAKE + 2), ALIGNMENT), (dict(D=FAKE + 2), ALIGNMENT), (dict(bias=FAKE + 2), ALIGNMENT)])
def test_scan_refusals(lib, kw, code):
    assert scan_codes(lib, scan(**kw)) == code


def test_scan_outputs_and_workspace(lib):
    s, dy = scan(), dwc.Rows(FAKE, 40, 8)
    fwd = lambda state=FAKE, y=FAKE, last=FAKE, saved=FAKE: lib.dwc_selective_scan_fwd(  # noqa: E731
        s, state, y, last, saved, FAKE, 1 << 30, None)
    assert fwd(y=None) == INVALID
    for k in ("state", "last", "saved"):
        assert fwd(**{k: FAKE + 2}) == ALIGNMENT
    need = lib.dwc_selective_scan_bwd_workspace_size(s)
    assert need > 0 and lib.dwc_selective_scan_bwd_workspace_size(scan(N=129)) == 0
    assert lib.dwc_selective_scan_saved_floats(s) == 2 * 8 * 4 and lib.dwc_selective_scan_saved_floats(scan(length=33)) == 6 * 8 * 4

    def bwd(**kw):
        a = dict(dy=dy, saved=FAKE, dfinal=None, du=FAKE, ddt=FAKE, dz=FAKE, db=FAKE, dc=FAKE, dA=FAKE, dD=FAKE, bias=FAKE,
                 dstate=FAKE, ws=FAKE, n=need)
        a.update(kw)
        return lib.dwc_selective_scan_bwd(s, *a.values(), None)

    for k in ("dy", "saved", "du", "ddt", "dz", "db", "dc", "dA", "dD", "bias"):
        assert bwd(**{k: None}) == INVALID, k
    for k in ("saved", "dfinal", "du", "dA", "dD", "bias", "dstate"):
        assert bwd(**{k: FAKE + 2}) == ALIGNMENT, k
    assert bwd(ws=None) == WORKSPACE and bwd(n=need - 1) == WORKSPACE and bwd(ws=FAKE + 4) == ALIGNMENT


def test_scan_step_refusals(lib):
    step = lambda s, state=FAKE, stride=32, y=FAKE: lib.dwc_selective_scan_step(s, state, stride, y, None)  # noqa: E731
    assert step(scan()) == INVALID and step(scan(length=1, offsets=FAKE)) == INVALID
    one = scan(length=1)
    assert step(one, stride=31) == INVALID and step(one, state=None) == INVALID and step(one, y=None) == INVALID
    assert step(one, state=FAKE + 2) == ALIGNMENT and step(one, stride=1 << 40) == UNSUPPORTED


def test_zero_beside_refusals(lib):
    def call(seqs=None, p=FAKE, n=64, count=1):
        return lib.dwc_zero_beside_sequences(seqs or dwc.Seqs(2, 8, FAKE), (ctypes.c_void_p * 1)(p), (ctypes.c_longlong * 1)(n), count,
                                             None)
    assert call(p=None) == INVALID and call(n=-2) == INVALID and call(count=-1) == INVALID and call(count=9) == UNSUPPORTED
    assert call(n=3) == ALIGNMENT and call(p=FAKE + 1) == ALIGNMENT and call(dwc.Seqs(0, 8, FAKE)) == INVALID
    assert call(dwc.Seqs(2, 8, None)) == 0


def norm_fwd(lib, x=FAKE, ldx=16, res=2 * FAKE, ldres=16, gate=3 * FAKE, ldgate=16, act=2, post=FAKE, pre=FAKE, scale=FAKE, pt=0,
             alpha=1.0, eps=1e-5, z=4 * FAKE, y=5 * FAKE, rpost=FAKE, rpre=FAKE, rows=4, C=16, dt=0, rt=0):
    return lib.dwc_block_norm_fwd(x, ldx, res, ldres, gate, ldgate, act, post, pre, scale, pt, alpha, eps, z, y, rpost, rpre, rows, C,
                                  dt, rt, None)


def norm_bwd(lib, dy=FAKE, lddy=16, dz=2 * FAKE, lddz=16, x=3 * FAKE, ldx=16, z=4 * FAKE, ldz=16, gate=5 * FAKE, ldgate=16, act=2,
             rpost=FAKE, rpre=FAKE, post=FAKE, pre=FAKE, scale=FAKE, pt=0, alpha=1.0, dx=6 * FAKE, dres=7 * FAKE, dgate=8 * FAKE,
             g0=FAKE, g1=FAKE, g2=FAKE, rows=4, C=16, dt=0, rt=0, ws=FAKE, nws=1 << 20):
    return lib.dwc_block_norm_bwd(dy, lddy, dz, lddz, x, ldx, z, ldz, gate, ldgate, act, rpost, rpre, post, pre, scale, pt, alpha, dx,
                                  dres, dgate, g0, g1, g2, rows, C, dt, rt, ws, nws, None)


@pytest.mark.parametrize("call", [norm_fwd, norm_bwd])
@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID), (dict(C=0), INVALID), (dict(dt=7), INVALID), (dict(rt=1), INVALID), (dict(dt=1, rt=2), INVALID),
    (dict(pt=3), INVALID), (dict(act=3), INVALID), (dict(act=-1), INVALID), (dict(alpha=float("inf")), INVALID), (dict(x=None), INVALID),
    (dict(z=None), INVALID), (dict(ldx=15), INVALID), (dict(ldgate=15), INVALID), (dict(C=(1 << 24) + 1), UNSUPPORTED),
    (dict(rows=1 << 37), UNSUPPORTED), (dict(ldx=1 << 39), UNSUPPORTED), (dict(x=FAKE + 2), ALIGNMENT), (dict(gate=FAKE + 2), ALIGNMENT),
    (dict(post=FAKE + 2), ALIGNMENT), (dict(pre=FAKE + 2), ALIGNMENT), (dict(scale=FAKE + 1, pt=1), ALIGNMENT),
    (dict(rpost=FAKE + 2), ALIGNMENT), (dict(rows=0), 0)])
def test_block_norm_refusals(lib, call, kw, code):
    if kw == dict(rows=0) and call is norm_bwd:
        kw = dict(rows=0, g0=None, g1=None, g2=None)
    assert call(lib, **kw) == code


def test_block_norm_outputs(lib):
    for kw in (dict(res=None), dict(y=None), dict(eps=-1.0), dict(eps=float("nan")), dict(z=FAKE, rt=0, dt=1, x=FAKE),
               dict(z=2 * FAKE, ldres=17)):
        assert norm_fwd(lib, **kw) == INVALID, kw
    for kw in (dict(dy=None), dict(dx=None), dict(dres=None), dict(rpost=None), dict(rpre=None), dict(gate=None), dict(dres=2 * FAKE, lddz=17)):
        assert norm_bwd(lib, **kw) == INVALID, kw
    assert norm_bwd(lib, ws=None) == WORKSPACE and norm_bwd(lib, nws=10) == WORKSPACE and norm_bwd(lib, ws=FAKE + 8) == ALIGNMENT
    assert norm_bwd(lib, g1=FAKE + 2) == ALIGNMENT and lib.dwc_block_norm_bwd_workspace_size(4, 0) == 0


def test_structures_match_the_header():
    assert (ctypes.sizeof(dwc.Rows), ctypes.sizeof(dwc.Seqs), ctypes.sizeof(dwc.CausalConv), ctypes.sizeof(dwc.Scan)) == (24, 24, 96, 192)


def test_the_binding_refuses_cpu_tensors():
    x, w = torch.zeros(2, 3, 8), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="no CPU fallback"):
        dwc.causal_conv_fwd(x, w)
    with pytest.raises(ValueError, match="no CPU fallback"):
        dwc.selective_scan_fwd(x, x, torch.zeros(8, 4), torch.zeros(2, 3, 4), torch.zeros(2, 3, 4))
    with pytest.raises(ValueError, match="no CPU fallback"):
        dwc.block_norm_fwd(x, x)
    with pytest.raises(TypeError):
        dwc.causal_conv_fwd(None, w)
