"""Layer norm, dropout and their residual form on the GPU against the fp64 definitions in
oracle/norm.py, element by element within that module's derived bounds: every type pair, channel
counts around the kernels' vector, warp and CTA limits, few and many rows, strided and unaligned
views, updates in place, other streams, graphs, offsets past 32 bits, infinities and NaN."""
import numpy as np
import pytest
import torch

import depthwise_convolution_nhwc_gb300 as dwc
from oracle import norm as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# (stream: layer norm's x, the residual and its sum; branch: y, the residual form's x, dy)
PAIRS = [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("f32", "f16")]
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dwc.build()
    dwc.load_library()
    yield
    assert dwc.device_status() == 0, "a kernel reported a timed-out wait"


def d(t):
    return t.detach().double().cpu().numpy()


def rand(rng, shape, dtype, scale=1.0, centre=0.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale + centre).to(DT[dtype])


def inputs(rows, C, wide, narrow, seed, gdt="f32"):
    """Rows with their own means, channels with their own spreads, one channel far out."""
    rng = np.random.default_rng(seed)
    spread = np.exp(0.3 * rng.standard_normal(C))
    spread[C // 2] *= 20
    s = {"z": torch.from_numpy(rng.standard_normal((rows, C)) * spread + rng.standard_normal((rows, 1))).to(DT[wide]),
         "x": rand(rng, (rows, C), narrow, 0.7), "dy": rand(rng, (rows, C), narrow, 0.5),
         "dz": rand(rng, (rows, C), wide, 0.5), "gamma": rand(rng, C, gdt, 0.3, 1.0), "beta": rand(rng, C, gdt, 0.3)}
    return {k: v.cuda() for k, v in s.items()}


def within(got, want, bound, what):
    got = d(got)
    assert got.shape == want.shape, what
    off = np.abs(got - want)
    assert np.all(off <= bound), (f"{what}: {np.sum(~(off <= bound))} of {off.size} outside, worst "
                                  f"{np.nanmax(off / np.maximum(bound, 1e-300)):.3g} of the bound")


def check_ln(s, wide, narrow, gamma=True, beta=True):
    g, b = (s["gamma"] if gamma else None), (s["beta"] if beta else None)
    gn, bn = (d(g) if gamma else 1.0), (d(b) if beta else 0.0)
    C = s["z"].shape[-1]
    z, dy = d(s["z"]).reshape(-1, C), d(s["dy"]).reshape(-1, C)
    y, mean, rstd = dwc.layer_norm_fwd(s["z"], g, b, EPS, out_dtype=DT[narrow], stats=True)
    want = ref.layer_norm(z, gn, bn, EPS)
    bound = ref.layer_norm_bound(z, gn, bn, EPS, narrow)
    within(y.reshape(-1, C), want[0], bound[0], "y")
    within(mean.reshape(-1), want[1], bound[1], "mean")
    within(rstd.reshape(-1), want[2], bound[2], "rstd")
    assert torch.equal(dwc.layer_norm_fwd(s["z"], g, b, EPS, out_dtype=DT[narrow]), y)
    m, r = d(mean).reshape(-1), d(rstd).reshape(-1)
    got = dwc.layer_norm_bwd(s["dy"], s["z"], mean, rstd, g)
    assert got[0].dtype == DT[wide] and got[1].dtype == got[2].dtype == torch.float32
    want, bound = ref.layer_norm_bwd(dy, z, m, r, gn), ref.layer_norm_bwd_bound(dy, z, m, r, gn, wide)
    for name, a, w, e in zip(("dx", "dgamma", "dbeta"), got, want, bound):
        within(a.reshape(w.shape), w, e, name)
    only = dwc.layer_norm_bwd(s["dy"], s["z"], mean, rstd, g, param_grads=False)
    assert only[1] is None and only[2] is None and torch.equal(only[0], got[0])


def check_add(s, wide, narrow, p, seed=11, offset=3, dz=True, inplace=False):
    gn, bn = d(s["gamma"]), d(s["beta"])
    C = s["z"].shape[-1]
    x, res, dy, dzn = (d(s[k]).reshape(-1, C) for k in ("x", "z", "dy", "dz"))
    u = ref.U["f32"]
    dropped = ref.dropout(x, p, seed, offset)
    zsum = res + dropped
    e_z = 2 * u * np.abs(dropped) + u * np.abs(zsum)
    stream = s["z"].clone()
    y, z, mean, rstd = dwc.add_layer_norm_fwd(s["x"], stream, s["gamma"], s["beta"], EPS, p, seed, offset, stats=True,
                                              z=stream if inplace else None)
    if not inplace:
        assert torch.equal(stream.nan_to_num(), s["z"].nan_to_num())
    assert y.dtype == DT[narrow] and z.dtype == DT[wide]
    within(z.reshape(-1, C), zsum, 1.01 * (e_z + ref.U[wide] * np.abs(zsum)) + ref.TINY[wide], "z")
    want = ref.layer_norm(zsum, gn, bn, EPS)
    bound = ref.layer_norm_bound(zsum, gn, bn, EPS, narrow, e_z)
    want_y, bound_y = want[0], bound[0]
    within(y.reshape(-1, C), want_y, bound_y, "y")
    within(mean.reshape(-1), want[1], bound[1], "mean")
    within(rstd.reshape(-1), want[2], bound[2], "rstd")
    # (a dense copy, as above: another row stride may take another kernel and order of sums)
    y2, z2 = dwc.add_layer_norm_fwd(s["x"], s["z"].clone(), s["gamma"], s["beta"], EPS, p, seed, offset)
    assert torch.equal(y, y2) and torch.equal(z, z2)

    zd, m, r = d(z).reshape(-1, C), d(mean).reshape(-1), d(rstd).reshape(-1)
    g, dgamma, dbeta = ref.layer_norm_bwd(dy, zd, m, r, gn)
    e_g, e_gamma, e_beta = ref.layer_norm_bwd_bound(dy, zd, m, r, gn, "f32", dzn if dz else None)
    if dz:
        g = g + dzn
    if not s["z"].is_contiguous():
        y2, z2 = dwc.add_layer_norm_fwd(s["x"], s["z"], s["gamma"], s["beta"], EPS, p, seed, offset)
        within(y2.reshape(-1, C), want_y, bound_y, "y of a strided stream")
        assert torch.equal(z, z2)
    got = dwc.add_layer_norm_bwd(s["dy"], z, mean, rstd, s["gamma"], s["dz"] if dz else None, p, seed, offset)
    within(got[1].reshape(-1, C), g, 1.01 * (e_g + ref.U[wide] * np.abs(g)) + ref.TINY[wide], "dres")
    dx = ref.dropout(g, p, seed, offset)
    scale = ref.dropout(np.ones_like(g), p, seed, offset)
    within(got[0].reshape(-1, C), dx, 1.01 * (scale * e_g + (2 * u + ref.U[narrow]) * np.abs(dx)) +
           (scale != 0) * ref.TINY[narrow], "dx")
    if p == 0.0 and wide == narrow:
        assert got[0] is got[1]
    within(got[2], dgamma, e_gamma, "dgamma")
    within(got[3], dbeta, e_beta, "dbeta")


# Around vectors (8 elements), lane groups (64, 128, 256 channels), a warp's most (1024) and a
# CTA's; odd counts and multiples of 8.
CHANNELS = [1, 2, 3, 7, 8, 9, 31, 32, 33, 56, 64, 65, 96, 100, 127, 128, 129, 192, 250, 256, 257, 384, 511, 512, 513,
            768, 1000, 1001, 1024, 1025, 1032, 2047, 2048, 2056, 4095, 4096, 4104, 5000, 8191, 8192, 8200]
WIDE = [12289, 16384, 16392, 20001, 32768, 40000, 65536, 70001]


@pytest.mark.parametrize("pair", PAIRS, ids="-".join)
@pytest.mark.parametrize("C", CHANNELS)
def test_layer_norm(C, pair):
    rows = {0: 1, 1: 37, 2: 200}[C % 3]
    check_ln(inputs(rows, C, *pair, seed=C), *pair)


@pytest.mark.parametrize("pair", PAIRS, ids="-".join)
@pytest.mark.parametrize("C", CHANNELS)
def test_add_layer_norm(C, pair):
    rows = {0: 200, 1: 1, 2: 37}[C % 3]
    check_add(inputs(rows, C, *pair, seed=C + 1), *pair, p=(0.0, 0.1, 0.5)[C // 3 % 3], dz=C % 5 != 0,
              inplace=C % 2 == 0)


@pytest.mark.parametrize("pair", PAIRS, ids="-".join)
@pytest.mark.parametrize("C", WIDE)
def test_wide_rows(C, pair):
    s = inputs(5, C, *pair, seed=C)
    check_ln(s, *pair)
    check_add(s, *pair, p=0.2)


@pytest.mark.parametrize("pair", PAIRS, ids="-".join)
@pytest.mark.parametrize("rows,C", [(50176, 64), (20001, 96), (30000, 33), (9000, 257), (4000, 1000), (3000, 2048),
                                    (1300, 5003), (700, 8192)])
def test_many_rows(rows, C, pair):
    s = inputs(rows, C, *pair, seed=rows)
    check_ln(s, *pair)
    check_add(s, *pair, p=0.1)


@pytest.mark.parametrize("p", [1.0, 0.9999, 2.0 ** -16, 2.0 ** -18])
@pytest.mark.parametrize("C", [40, 1001, 2048])
def test_extreme_probabilities_of_the_residual_form(C, p):
    check_add(inputs(37, C, "f32", "f32", seed=C), "f32", "f32", p=p)


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 8, 9, 151, 152, 153, 304, 305, 609])
@pytest.mark.parametrize("C", [72, 1001, 2048])
def test_row_counts(rows, C):
    s = inputs(rows, C, "f32", "bf16", seed=rows)
    check_ln(s, "f32", "bf16")
    check_add(s, "f32", "bf16", p=0.3)


@pytest.mark.parametrize("rows", [11, 31, 32, 64, 100, 255, 256, 257])
@pytest.mark.parametrize("C", [8, 40, 65, 513, 1000, 4099, 5120, 8200])
def test_few_rows(rows, C):
    """Around the rules for calls of few rows: one CTA, columns added up in the row kernel, partial sums."""
    s = inputs(rows, C, "bf16", "bf16", seed=rows + C)
    check_ln(s, "bf16", "bf16")
    check_add(s, "bf16", "bf16", p=0.3, dz=rows % 2 == 0)


@pytest.mark.parametrize("gdt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gamma,beta", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("C", [100, 2048])
def test_parameters(C, gamma, beta, gdt):
    check_ln(inputs(19, C, "bf16", "bf16", seed=4, gdt=gdt), "bf16", "bf16", gamma, beta)


@pytest.mark.parametrize("pair", PAIRS, ids="-".join)
@pytest.mark.parametrize("shape,view", [
    ((40, 300), lambda t: t[:, 16:272]),           # aligned channels of wider rows
    ((40, 300), lambda t: t[:, 5:205]),            # unaligned ones
    ((40, 2056), lambda t: t[:, 1:2050]),
    ((4, 21, 64), lambda t: t[:, ::2].transpose(0, 1)[3]),   # every other token of one position
    ((33, 128), lambda t: t[::3]),
    ((33, 129), lambda t: t[1:]),                  # rows whose start is not aligned
    ((3, 5, 7, 96), lambda t: t),
    ((1000,), lambda t: t[3:]),
], ids=range(8))
def test_views(shape, view, pair):
    wide, narrow = pair
    rng = np.random.default_rng(9)
    s = {k: view(rand(rng, shape, dt, 1.0, 0.2).cuda()) for k, dt in (("z", wide), ("x", narrow), ("dy", narrow), ("dz", wide))}
    C = s["z"].shape[-1]
    s["gamma"], s["beta"] = rand(rng, C, "f32", 0.3, 1.0).cuda(), rand(rng, C, "f32", 0.3).cuda()
    check_ln(s, wide, narrow)
    check_add(s, wide, narrow, p=0.25)
    # one dense operand among strided ones
    s["dy"], s["x"] = s["dy"].contiguous(), s["x"].contiguous()
    check_ln(s, wide, narrow)
    check_add(s, wide, narrow, p=0.25)


def test_outputs_stay_inside_their_rows():
    """Outputs in the middle of a larger buffer leave its other elements alone."""
    for C in (33, 64, 1001, 4096, 9001):
        for lead in (0, 1, 8):
            buf = torch.full((lead + 5 * C + 24,), 7.0, device="cuda", dtype=torch.bfloat16)
            out = buf[lead:lead + 5 * C].view(5, C)
            x = torch.randn(5, C, device="cuda").bfloat16()
            dwc.layer_norm_fwd(x, out=out)
            within(out, ref.layer_norm(d(x), 1.0, 0.0, EPS)[0], ref.layer_norm_bound(d(x), 1.0, 0.0, EPS, "bf16")[0],
                   (C, lead))
            dwc.dropout_fwd(x, 0.5, 1, out=out)
            assert torch.equal(out, dwc.dropout_fwd(x, 0.5, 1)), (C, lead)
            assert bool((buf[:lead] == 7).all()) and bool((buf[lead + 5 * C:] == 7).all()), (C, lead)


# ----------------------------------------------------------------------------- extremes

def test_rows_of_equal_values():
    x = torch.full((3, 200), 100.0, device="cuda")
    x[1] = 0.0
    beta = torch.linspace(-1, 1, 200, device="cuda")
    y, mean, rstd = dwc.layer_norm_fwd(x, None, beta, EPS, stats=True)
    b = ref.layer_norm_bound(d(x), 1.0, d(beta), EPS, "f32")
    within(y, np.broadcast_to(d(beta), (3, 200)), b[0], "y")
    assert torch.equal(mean, torch.tensor([100.0, 0.0, 100.0], device="cuda"))
    # eps = 0 and no spread: 0 * infinity, as the formula has it; a single channel likewise
    assert dwc.layer_norm_fwd(x[1:2], eps=0.0).isnan().all()
    assert torch.equal(dwc.layer_norm_fwd(torch.randn(9, 1, device="cuda")), torch.zeros(9, 1, device="cuda"))


@pytest.mark.parametrize("C", [64, 1000, 4096, 20000])
def test_far_mean_keeps_its_precision(C):
    """A mean 3000 times the spread: squares of the values themselves would lose the variance."""
    rng = np.random.default_rng(C)
    x = torch.from_numpy(3000 + rng.standard_normal((7, C))).float().cuda()
    y, mean, rstd = dwc.layer_norm_fwd(x, stats=True)
    want, bound = ref.layer_norm(d(x), 1.0, 0.0, EPS), ref.layer_norm_bound(d(x), 1.0, 0.0, EPS, "f32")
    for a, w, b in zip((y, mean, rstd), want, bound):
        within(a, w, b, "far mean")
    assert np.max(np.abs(d(rstd) / want[2] - 1)) < 0.02


@pytest.mark.parametrize("C", [40, 512, 3000])
def test_infinities_and_nan_stay_in_their_rows(C):
    s = inputs(33, C, "f32", "f32", seed=5)
    clean = dwc.layer_norm_fwd(s["z"], s["gamma"], s["beta"])
    z = s["z"].clone()
    z[4, 7], z[20, C - 1], z[32, 0] = float("inf"), float("nan"), float("-inf")
    y, mean, rstd = dwc.layer_norm_fwd(z, s["gamma"], s["beta"], stats=True)
    bad = [4, 20, 32]
    good = [r for r in range(33) if r not in bad]
    assert y[bad].isnan().all() and torch.equal(y[good], clean[good])
    dx, dgamma, dbeta = dwc.layer_norm_bwd(s["dy"], z, mean, rstd, s["gamma"])
    assert dx[bad].isnan().all() and dx[good].isfinite().all()
    assert dgamma.isnan().all() and dbeta.isfinite().all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_dropped_infinities_and_nan_give_zero(dtype):
    n, seed = 1003, 77
    keep = ref.kept(0, n, 0.6, seed, 0)
    x = torch.full((1, n), float("nan"), device="cuda", dtype=DT[dtype])
    x[0, ::2] = float("inf")
    x[0, ::3] = torch.finfo(DT[dtype]).min
    y = d(dwc.dropout_fwd(x, 0.6, seed))[0]
    assert np.all(y[~keep] == 0) and not np.signbit(y[~keep]).any()
    assert not np.any(y[keep] == 0)
    assert (d(dwc.dropout_fwd(x, 1.0, seed)) == 0).all()
    z = torch.zeros(1, n, device="cuda", dtype=DT[dtype])
    _, zs = dwc.add_layer_norm_fwd(x, z, p=0.6, seed=seed)
    assert np.all(d(zs)[0][~keep] == 0)


def test_no_rows():
    x = torch.empty(0, 16, device="cuda")
    y, mean, rstd = dwc.layer_norm_fwd(x, stats=True)
    assert y.shape == (0, 16) and mean.shape == (0,)
    dx, dgamma, dbeta = dwc.layer_norm_bwd(x, x, mean, rstd)
    assert dx.shape == (0, 16) and (dgamma == 0).all() and (dbeta == 0).all()
    assert dwc.dropout_fwd(x, 0.1, 1).shape == (0, 16)
    assert dwc.add_layer_norm_fwd(x, x)[0].shape == (0, 16)


# ------------------------------------------------------------------------------ dropout

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (1, 8), (3, 5), (17, 33), (4, 1000), (9, 1001), (301, 520), (2, 3, 4, 64),
                                   (100003,), (70, 4096)])
@pytest.mark.parametrize("p", [0.0, 1e-9, 0.1, 0.5, 0.999, 1.0])
def test_dropout(shape, p, dtype):
    rng = np.random.default_rng(1)
    x = rand(rng, shape, dtype).cuda()
    seed, offset = 2 ** 63 + 12345, 2 ** 40 + 1
    want = ref.dropout(d(x), p, seed, offset)
    y = dwc.dropout_fwd(x, p, seed, offset)
    within(y, want, 1.01 * (2 * ref.U["f32"] + ref.U[dtype]) * np.abs(want) + (want != 0) * ref.TINY[dtype], "y")
    assert np.array_equal(d(y) == 0, want == 0) or dtype == "f16"
    assert torch.equal(dwc.dropout_bwd(x, p, seed, offset), y)
    if p < 2 ** -17:
        assert torch.equal(y, x)
    dwc.dropout_fwd(x, p, seed, offset, out=x)
    assert torch.equal(x, y)


def test_dropout_of_views_counts_logical_elements():
    t = torch.randn(50, 200, device="cuda")
    for v in (t[:, 3:100], t[::2, 8:136], t[:, 7:8]):
        assert torch.equal(dwc.dropout_fwd(v, 0.3, 5), dwc.dropout_fwd(v.contiguous(), 0.3, 5))
    t = torch.randn(301, 1072, device="cuda")
    for dt in DT.values():
        u = t.to(dt)
        for v in (u[:, :8], u[:, 16:1064], u[3:, 64:128], u[::3, 8:1048], u[7:8, 8:64], u[:, 8:13], u[:, :1071]):
            assert torch.equal(dwc.dropout_fwd(v, 0.3, 5, 2), dwc.dropout_fwd(v.contiguous(), 0.3, 5, 2))


def test_offsets_past_32_bits():
    """2^32 + a ragged tail of elements: counters, addresses and rows past 32 bits."""
    C, rows = 8200, (1 << 32) // 8200 + 3
    first = (rows - 2) * C
    assert first > 1 << 32
    x = torch.empty(rows, C, device="cuda", dtype=torch.bfloat16).fill_(1.0)
    tail = torch.randn(2, C, device="cuda").bfloat16()
    x[-2:] = tail
    want = ref.dropout(d(tail), 0.2, 9, 1, first=first)
    y = dwc.dropout_fwd(x, 0.2, 9, 1)
    within(y[-2:], want, 1.01 * (2 * ref.U["f32"] + ref.U["bf16"]) * np.abs(want), "dropout tail")
    y, mean, rstd = dwc.layer_norm_fwd(x, out=y, stats=True)
    w, b = ref.layer_norm(d(tail), 1.0, 0.0, EPS), ref.layer_norm_bound(d(tail), 1.0, 0.0, EPS, "bf16")
    within(y[-2:], w[0], b[0], "y tail")
    y2, z = dwc.add_layer_norm_fwd(x, x, p=0.2, seed=9, offset=1, out=y)
    zs = d(tail) + want
    within(z[-2:], zs, 1.01 * ref.U["bf16"] * np.abs(zs) + 1e-6, "z tail")
    dx, dgamma, _ = dwc.layer_norm_bwd(x, x, mean, rstd, out=y)
    m, r = d(mean[-2:]), d(rstd[-2:])
    w = ref.layer_norm_bwd(d(tail), d(tail), m, r, 1.0)
    b = ref.layer_norm_bwd_bound(d(tail), d(tail), m, r, 1.0, "bf16")
    within(dx[-2:], w[0], b[0], "dx tail")


# ------------------------------------------------------------- gradients against differences

@pytest.mark.parametrize("C", [48, 1001, 4096])
def test_gradient_along_a_direction(C):
    """(L(+h) - L(-h)) / 2h of L = sum(y dy) + sum(z dz) with the kernels' own fp32 forward pass,
    summed in 64 bits, against the kernels' gradients.  At h = 2^-5 the truncation is below
    h^2 of the derivative's scale (1e-3), the rounding sqrt(n) 1e-7 / h near 1e-5 of it; the scale is
    the product of the norms over sqrt(n)."""
    s, p, h = inputs(24, C, "f32", "f32", seed=C), 0.3, 2.0 ** -5
    rng = np.random.default_rng(8)

    def loss(x, res, gamma, beta):
        y, z = dwc.add_layer_norm_fwd(x, res, gamma, beta, EPS, p, 3, 1)
        return float((y.double() * s["dy"].double()).sum() + (z.double() * s["dz"].double()).sum())

    args = [s["x"], s["z"], s["gamma"], s["beta"]]
    _, z, mean, rstd = dwc.add_layer_norm_fwd(*args, EPS, p, 3, 1, stats=True)
    grads = dwc.add_layer_norm_bwd(s["dy"], z, mean, rstd, s["gamma"], s["dz"], p, 3, 1)
    for k, g in enumerate(grads):
        v = torch.from_numpy(rng.standard_normal(tuple(args[k].shape))).float().cuda()
        moved = [[a + sign * h * v if i == k else a for i, a in enumerate(args)] for sign in (1, -1)]
        got = (loss(*moved[0]) - loss(*moved[1])) / (2 * h)
        want = float((g.double() * v.double()).sum())
        scale = float(g.double().norm() * v.double().norm()) / np.sqrt(v.numel()) + float(s["dy"].double().norm())
        assert abs(got - want) < 5e-3 * scale, (k, got, want, scale)


# ----------------------------------------------------------------------- streams and graphs

def test_results_repeat_bit_for_bit():
    for C in (96, 1001, 4096):
        s = inputs(3001, C, "bf16", "bf16", seed=2)
        first = dwc.add_layer_norm_fwd(s["x"], s["z"], s["gamma"], s["beta"], EPS, 0.1, 4, 4, stats=True)
        back = dwc.add_layer_norm_bwd(s["dy"], first[1], first[2], first[3], s["gamma"], s["dz"], 0.1, 4, 4)
        for _ in range(5):
            again = dwc.add_layer_norm_fwd(s["x"], s["z"], s["gamma"], s["beta"], EPS, 0.1, 4, 4, stats=True)
            b2 = dwc.add_layer_norm_bwd(s["dy"], first[1], first[2], first[3], s["gamma"], s["dz"], 0.1, 4, 4)
            assert all(torch.equal(a, b) for a, b in zip(first + back, again + b2))


def test_calls_on_another_stream():
    s = inputs(4000, 512, "f32", "f32", seed=6)
    want = dwc.layer_norm_fwd(s["z"], s["gamma"], s["beta"], stats=True)
    wantb = dwc.layer_norm_bwd(s["dy"], s["z"], want[1], want[2], s["gamma"])
    torch.cuda.synchronize()
    side, both = torch.cuda.Stream(), []
    for _ in range(20):
        both.append(dwc.layer_norm_bwd(s["dy"], s["z"], want[1], want[2], s["gamma"], stream=side))
        both.append(dwc.layer_norm_bwd(s["dy"], s["z"], want[1], want[2], s["gamma"]))
    got = dwc.layer_norm_fwd(s["z"], s["gamma"], s["beta"], stats=True, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for r in both for a, b in zip(r, wantb))


def test_back_to_back_calls_see_each_other():
    """A chain of dependent launches without anything between them."""
    s = inputs(2000, 256, "f32", "f32", seed=3)
    x = s["z"]
    for k in range(30):
        x = dwc.dropout_fwd(dwc.layer_norm_fwd(x, s["gamma"], s["beta"]), 0.01, 5, k)
    y = s["z"]
    for k in range(30):
        y = dwc.layer_norm_fwd(y, s["gamma"], s["beta"])
        torch.cuda.synchronize()
        y = dwc.dropout_fwd(y, 0.01, 5, k)
        torch.cuda.synchronize()
    assert torch.equal(x, y)


@pytest.mark.parametrize("C", [1024, 1001, 12288])
def test_graph_draws_new_masks_as_its_step_advances(C):
    s = inputs(64, C, "bf16", "bf16", seed=3)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    stats = dwc.layer_norm_fwd(s["z"], stats=True)[1:]

    def work():
        y, z = dwc.add_layer_norm_fwd(s["x"], s["z"], s["gamma"], s["beta"], EPS, 0.5, 9, step)
        dx = dwc.add_layer_norm_bwd(s["dy"], s["z"], *stats, s["gamma"], None, 0.5, 9, step)[0]
        return y, z, dx, dwc.dropout_fwd(s["x"], 0.5, 9, step)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for k in (0, 1, 2 ** 33):
        step.fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        y, z = dwc.add_layer_norm_fwd(s["x"], s["z"], s["gamma"], s["beta"], EPS, 0.5, 9, k)
        dx = dwc.add_layer_norm_bwd(s["dy"], s["z"], *stats, s["gamma"], None, 0.5, 9, k)[0]
        for a, b in zip(out, (y, z, dx, dwc.dropout_fwd(s["x"], 0.5, 9, k))):
            assert torch.equal(a, b), k


# ------------------------------------------------------------------------------ refusals

def test_binding_refusals():
    x = torch.randn(6, 32, device="cuda")
    st = torch.zeros(6, device="cuda")
    h = x.half()
    bad = [
        lambda: dwc.layer_norm_fwd(x.t()), lambda: dwc.layer_norm_fwd(x[:, ::2]),
        lambda: dwc.layer_norm_fwd(x[:1].expand(6, 32)), lambda: dwc.layer_norm_fwd(x, torch.ones(31, device="cuda")),
        lambda: dwc.layer_norm_fwd(x, torch.ones(32)), lambda: dwc.layer_norm_fwd(x, torch.ones(32, device="cuda"), torch.ones(32, device="cuda").half()),
        lambda: dwc.layer_norm_fwd(x, out=torch.empty(6, 33, device="cuda")), lambda: dwc.layer_norm_fwd(x, out=torch.empty(32, 6, device="cuda").t()),
        lambda: dwc.layer_norm_bwd(x[:5], x, st, st), lambda: dwc.layer_norm_bwd(x, x, st[:5], st),
        lambda: dwc.layer_norm_bwd(x, x, st.double(), st), lambda: dwc.layer_norm_fwd(torch.empty(4, 0, device="cuda")),
        lambda: dwc.dropout_fwd(x, 1.5, 1), lambda: dwc.dropout_fwd(x, -0.1, 1), lambda: dwc.dropout_fwd(x, float("nan"), 1),
        lambda: dwc.dropout_fwd(x, 0.1, 1, torch.zeros(1, device="cuda")), lambda: dwc.dropout_fwd(x, 0.1, 1, torch.zeros(1, dtype=torch.int64)),
        lambda: dwc.add_layer_norm_fwd(x, x[:5]), lambda: dwc.add_layer_norm_fwd(x, x, z=h),
        lambda: dwc.add_layer_norm_bwd(x, x, st, st, dz=h),
    ]
    for k, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
    for k, f in enumerate((lambda: dwc.layer_norm_fwd(h, out_dtype=torch.float32), lambda: dwc.layer_norm_fwd(x, eps=-1.0),
                           lambda: dwc.add_layer_norm_fwd(x, h), lambda: dwc.add_layer_norm_fwd(h, h.bfloat16()),
                           lambda: dwc.layer_norm_bwd(x, h, st, st))):
        with pytest.raises(dwc.DwcError):
            f()
    with pytest.raises(TypeError):
        dwc.layer_norm_fwd(x.double())
    assert torch.isfinite(dwc.layer_norm_fwd(x)).all()
