"""Layer norm, dropout and their residual form without a GPU: the 64-bit definitions (gradients
against differences, the generator against its published vectors) and the refusals of the C ABI
and the binding."""
import os

import numpy as np
import pytest
import torch

import depthwise_convolution_nhwc_gb300 as dwc
from oracle import norm as ref

FAKE = 0x10000  # never dereferenced: every case below fails validation first
NAN = float("nan")


# ---------------------------------------------------------------------------- definitions

@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_generator_matches_the_published_vectors(counter, key, words):
    assert tuple(ref.philox4x32_10(counter, key)) == words


def test_mask_is_the_generator_element_by_element():
    seed, offset, p = 0x123456789ABCDEF0, 0xFEDCBA9876543210, 0.3
    q = int(np.floor(p * 65536 + 0.5))
    for first in (0, 5, 2 ** 35 - 3):
        got = ref.kept(first, 21, p, seed, offset)
        for n, i in enumerate(range(first, first + 21)):
            b = i // 8
            w = ref.philox4x32_10((b & 0xFFFFFFFF, b >> 32, offset & 0xFFFFFFFF, offset >> 32),
                                  (seed & 0xFFFFFFFF, seed >> 32))
            h = (w[i % 8 // 2] >> (16 * (i % 2))) & 0xFFFF
            assert bool(got[n]) == (h >= q)


@pytest.mark.parametrize("p", [0.1, 0.5, 0.9])
def test_kept_share_and_scale(p):
    n = 1 << 18
    q = np.floor(p * 65536 + 0.5) / 65536
    share = ref.kept(0, n, p, 7, 1).mean()
    assert abs(share - (1 - q)) < 6 * np.sqrt(q * (1 - q) / n)   # six standard deviations
    y = ref.dropout(np.ones((1, n)), p, 7, 1)
    assert set(np.unique(y)) == {0.0, 1 / (1 - q)}


def test_gradients_match_differences():
    """Central differences of sum(y * dy) + sum(z * dz) in 64 bits: truncation h^2 and rounding
    1e-16 / h are both near 1e-10 at h = 1e-5 for values and derivatives of order 1 to 10."""
    rng = np.random.default_rng(3)
    R, C, eps, p, seed = 3, 11, 1e-3, 0.4, 5
    x, res, dy, dz = (rng.standard_normal((R, C)) for _ in range(4))
    gamma, beta = 1 + 0.3 * rng.standard_normal(C), rng.standard_normal(C)

    def loss(x, res, gamma, beta):
        z = res + ref.dropout(x, p, seed, 2)
        return (ref.layer_norm(z, gamma, beta, eps)[0] * dy).sum() + (z * dz).sum()

    z = res + ref.dropout(x, p, seed, 2)
    _, mean, rstd = ref.layer_norm(z, gamma, beta, eps)
    g, dgamma, dbeta = ref.layer_norm_bwd(dy, z, mean, rstd, gamma)
    g = g + dz
    grads = [ref.dropout(g, p, seed, 2), g, dgamma, dbeta]
    args, h = [x, res, gamma, beta], 1e-5
    for k, want in enumerate(grads):
        got = np.empty_like(want)
        for i in np.ndindex(want.shape):
            side = []
            for s in (h, -h):
                moved = [a.copy() for a in args]
                moved[k][i] += s
                side.append(loss(*moved))
            got[i] = (side[0] - side[1]) / (2 * h)
        np.testing.assert_allclose(got, want, rtol=1e-6, atol=1e-7)


# ------------------------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dwc.LIB_PATH):
        dwc.build()
    return dwc.load_library()


def ln_fwd(lib, x=FAKE, ldx=16, gamma=FAKE, beta=FAKE, pt=0, eps=1e-5, y=FAKE, mean=FAKE, rstd=FAKE, rows=4,
           C=16, dt=0, od=0):
    return lib.dwc_layer_norm_fwd(x, ldx, gamma, beta, pt, eps, y, mean, rstd, rows, C, dt, od, None)


def ln_bwd(lib, dy=FAKE, lddy=16, x=FAKE, ldx=16, mean=FAKE, rstd=FAKE, gamma=FAKE, pt=0, dx=FAKE, dgamma=FAKE,
           dbeta=FAKE, rows=4, C=16, dt=0, dyt=0, ws=FAKE, nws=1 << 20):
    return lib.dwc_layer_norm_bwd(dy, lddy, x, ldx, mean, rstd, gamma, pt, dx, dgamma, dbeta, rows, C, dt, dyt,
                                  ws, nws, None)


def drop(lib, x=FAKE, ldx=16, y=FAKE, rows=4, C=16, p=0.1, seed=1, offset=0, step=None, dt=0):
    codes = {f(x, ldx, y, rows, C, p, seed, offset, step, dt, None)
             for f in (lib.dwc_dropout_fwd, lib.dwc_dropout_bwd)}
    assert len(codes) == 1
    return codes.pop()


def add_fwd(lib, x=FAKE, ldx=16, res=2 * FAKE, ldres=16, p=0.1, step=None, gamma=FAKE, beta=FAKE, pt=0, eps=1e-5,
            z=FAKE, y=FAKE, mean=FAKE, rstd=FAKE, rows=4, C=16, dt=0, rt=0):
    return lib.dwc_add_layer_norm_fwd(x, ldx, res, ldres, p, 1, 0, step, gamma, beta, pt, eps, z, y, mean, rstd,
                                      rows, C, dt, rt, None)


def add_bwd(lib, dy=FAKE, lddy=16, dz=FAKE, lddz=16, z=FAKE, ldz=16, mean=FAKE, rstd=FAKE, gamma=FAKE, pt=0, p=0.1,
            step=None, dx=FAKE, dres=FAKE, dgamma=FAKE, dbeta=FAKE, rows=4, C=16, dt=0, rt=0, ws=FAKE, nws=1 << 20):
    return lib.dwc_add_layer_norm_bwd(dy, lddy, dz, lddz, z, ldz, mean, rstd, gamma, pt, p, 1, 0, step, dx, dres,
                                      dgamma, dbeta, rows, C, dt, rt, ws, nws, None)


ALL = [ln_fwd, ln_bwd, drop, add_fwd, add_bwd]


@pytest.mark.parametrize("call", ALL)
def test_sizes_and_types_are_checked(lib, call):
    assert call(lib, rows=-1) == 1
    assert call(lib, C=0) == 1
    assert call(lib, dt=7) == 1
    assert call(lib, C=(1 << 24) + 1) == 2
    assert call(lib, rows=1 << 37) == 2
    ld = {ln_fwd: "ldx", ln_bwd: "lddy", drop: "ldx", add_fwd: "ldres", add_bwd: "ldz"}[call]
    assert call(lib, **{ld: 15}) == 1
    assert call(lib, **{ld: 1 << 39}) == 2


@pytest.mark.parametrize("call,pair", [(ln_fwd, ("dt", "od")), (ln_bwd, ("dt", "dyt")), (add_fwd, ("rt", "dt")),
                                       (add_bwd, ("rt", "dt"))])
def test_type_pairs(lib, call, pair):
    wide, narrow = pair
    for w, n in ((1, 0), (2, 0), (1, 2), (2, 1), (0, 5), (5, 0)):
        assert call(lib, **{wide: w, narrow: n}) == 1, (w, n)
    assert call(lib, pt=3) == 1
    assert call(lib, gamma=FAKE + 2) == 3 and call(lib, pt=1, gamma=FAKE + 1) == 3


@pytest.mark.parametrize("call,names", [(ln_fwd, ("x", "y")), (ln_bwd, ("dy", "x", "mean", "rstd", "dx")),
                                        (drop, ("x", "y")), (add_fwd, ("x", "res", "z", "y")),
                                        (add_bwd, ("dy", "z", "mean", "rstd", "dx", "dres"))])
def test_pointers(lib, call, names):
    for n in names:
        assert call(lib, **{n: None}) == 1, n
        assert call(lib, **{n: FAKE + 2}) == 3, n
    if call in (ln_fwd, add_fwd):
        assert call(lib, mean=FAKE + 2) == 3 and call(lib, beta=FAKE + 2) == 3
    if call in (ln_bwd, add_bwd):
        assert call(lib, dgamma=FAKE + 2) == 3


def test_eps_and_probability(lib):
    for call in (ln_fwd, add_fwd):
        for eps in (-1e-9, NAN, float("inf")):
            assert call(lib, eps=eps) == 1
    for call in (drop, add_fwd, add_bwd):
        for p in (-1e-9, 1.0001, NAN):
            assert call(lib, p=p) == 1
        assert call(lib, step=FAKE + 4) == 3


def test_updates_in_place_need_dense_rows(lib):
    assert add_fwd(lib, res=FAKE, z=FAKE, ldres=24) == 1
    assert drop(lib, x=FAKE, y=FAKE, ldx=24) == 1


def test_dx_may_be_left_out_only_where_it_is_dres(lib):
    assert add_bwd(lib, dx=None, p=0.1) == 1
    assert add_bwd(lib, dx=None, p=0.0, dt=1) == 1
    assert add_bwd(lib, dx=None, p=0.0, ws=None) == 4     # accepted as far as the workspace


def test_workspace(lib):
    need = lib.dwc_layer_norm_bwd_workspace_size(4, 16)
    assert need > 0
    for call in (ln_bwd, add_bwd):
        assert call(lib, ws=None) == 4
        assert call(lib, nws=need - 1) == 4
        assert call(lib, ws=FAKE + 4) == 3
    for rows, C in ((-1, 16), (4, 0), (0, 16), (4, (1 << 24) + 1)):
        assert lib.dwc_layer_norm_bwd_workspace_size(rows, C) == 0


def test_no_rows_is_no_work(lib):
    assert ln_fwd(lib, rows=0, x=None, y=None) == 0
    assert ln_bwd(lib, rows=0, dy=None, x=None, mean=None, rstd=None, dx=None, dgamma=None, dbeta=None) == 0
    assert drop(lib, rows=0, x=None, y=None) == 0
    assert add_fwd(lib, rows=0, x=None, res=None, z=None, y=None) == 0


def test_binding_takes_no_cpu_tensors():
    x, s = torch.zeros(4, 16), torch.zeros(4)
    for f in (lambda: dwc.layer_norm_fwd(x), lambda: dwc.layer_norm_bwd(x, x, s, s),
              lambda: dwc.dropout_fwd(x, 0.1, 1), lambda: dwc.dropout_bwd(x, 0.1, 1),
              lambda: dwc.add_layer_norm_fwd(x, x), lambda: dwc.add_layer_norm_bwd(x, x, s, s)):
        with pytest.raises(ValueError, match="no CPU fallback"):
            f()


@pytest.mark.parametrize("view,want", [
    (lambda t: t, 24), (lambda t: t[:, :, 3:11], 24), (lambda t: t[::2], None), (lambda t: t[:, 2:3], 120),
    (lambda t: t[1:2, ::2], 48), (lambda t: t[:, :, ::2], None), (lambda t: t.transpose(0, 1), None),
    (lambda t: t[0, 0], 24), (lambda t: t[:, :, :1], 24), (lambda t: t[:, :1, :1].expand(4, 5, 1), None),
    (lambda t: t[0, 0, ::2], None), (lambda t: t[0, 0, 5:6], 1),
])
def test_row_stride_of_views(view, want):
    from depthwise_convolution_nhwc_gb300.norm import _stride
    t = view(torch.zeros(4, 5, 24))
    if want is None:
        with pytest.raises(ValueError):
            _stride(t, "x")
    else:
        assert _stride(t, "x") == want
