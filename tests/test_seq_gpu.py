"""Causal convolution, selective scan and block norm on the GPU against the fp64 definitions in oracle/seq.py,
element by element within the bounds that come with them: types, channel, state and group counts, lengths around the
kernels' tiles, packed sequences (empty ones and rows beside them too), strided views, states carried on, single
tokens, other streams, graphs, infinities and NaN."""
import threading

import numpy as np
import pytest
import torch

import depthwise_convolution_nhwc_gb300 as dwc
from oracle import seq as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
NAMES = {v: k for k, v in DT.items()}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dwc.build()
    dwc.load_library()
    yield
    assert dwc.device_status() == 0, "a kernel reported a timed-out wait"


def d(t):
    return t.detach().double().cpu().numpy()


def rand(rng, shape, dtype, scale=1.0, centre=0.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale + centre).to(DT[dtype]).cuda()


def within(got, want, what):
    """`got` (a tensor) within the bound of `want` (a Val), rounded to got's type."""
    t = NAMES[got.dtype]
    got = d(got)
    assert got.shape == want.v.shape, (what, got.shape, want.v.shape)
    off, bound = np.abs(got - want.v), want.rounded(t)
    assert np.all(off <= bound), (f"{what}: {np.sum(~(off <= bound))} of {off.size} outside, worst "
                                  f"{np.nanmax(off / bound):.3g} of the bound")


def cat(list_, axis=0):
    return ref.Val(np.concatenate([x.v for x in list_], axis), np.concatenate([x.e for x in list_], axis))


def added(list_):
    return ref.stack(list_).sum(0)


def pieces(x, offsets):
    """The rows of every sequence."""
    if offsets is None:
        return [d(x[i]) for i in range(x.shape[0])]
    return [d(x[a:b]) for a, b in zip(offsets[:-1], offsets[1:])]


def joined(list_, offsets):
    return ref.stack(list_) if offsets is None else cat(list_)


def device(offsets):
    return None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")


def inside(t, offsets):
    """The packed rows that belong to sequences; those beside them must hold `beside`."""
    return t if offsets is None else t[offsets[0]:offsets[-1]]


# -------------------------------------------------------------------- causal convolution

def check_conv(rng, lead, C, K, dtype, act="silu", offsets=None, state=True, bias=True, pdt="f32", view=None, final=True):
    count = lead[0] if offsets is None else len(offsets) - 1
    view = view or (lambda shape: rand(rng, shape, dtype))
    x, dy = view((*lead, C)), view((*lead, C))
    w, b = rand(rng, (K, C), pdt, 0.7), rand(rng, C, pdt, 0.5) if bias else None
    s = rand(rng, (count, K - 1, C), dtype) if state else None
    df = rand(rng, (count, K - 1, C), dtype) if final else None
    off = device(offsets)
    got = dwc.causal_conv_fwd(x, w, b, act, s, off, final=final)
    y, last = got if final else (got, None)
    dx, dw, db, ds = dwc.causal_conv_bwd(dy, x, w, b, act, s, off, df)
    assert (ds is None) == (s is None) and (db is None) == (b is None)
    assert y.dtype == dx.dtype == x.dtype and y.is_contiguous() and dx.is_contiguous()
    xs, dys = pieces(x, offsets), pieces(dy, offsets)
    wn, bn = d(w), d(b) if bias else np.zeros(C)
    zero = np.zeros((K - 1, C))
    fwd = [ref.causal_conv(xs[i], wn, bn, act, d(s[i]) if state else zero) for i in range(count)]
    bwd = [ref.causal_conv_bwd(dys[i], xs[i], wn, bn, act, d(s[i]) if state else zero, d(df[i]) if final else zero, None)
           for i in range(count)]
    within(inside(y, offsets), joined([f[0] for f in fwd], offsets), "y")
    if final:
        assert torch.equal(last, torch.from_numpy(np.stack([f[1] for f in fwd])).to(last.dtype).cuda())
    within(inside(dx, offsets), joined([f[0] for f in bwd], offsets), "dx")
    within(dw, added([f[2] for f in bwd]), "dw")
    if bias:
        within(db, added([f[3] for f in bwd]), "dbias")
    if state:
        within(ds, ref.stack([f[1] for f in bwd]), "dstate")
    for t in (y, dx):
        if offsets is not None:
            assert not t[:offsets[0]].any() and not t[offsets[-1]:].any()
    only = dwc.causal_conv_bwd(dy, x, w, b, act, s, off, df, param_grads=False)
    assert torch.equal(only[0], dx) and only[1] is None and only[2] is None
    assert torch.equal(dwc.causal_conv_fwd(x, w, b, act, s, off), y)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 8, 16])
@pytest.mark.parametrize("C", [1, 8, 24, 33, 264])
def test_causal_conv(C, K, dtype):
    T = {0: 1, 1: 17, 2: 70}[(C + K) % 3]
    check_conv(np.random.default_rng(C * 31 + K), (3, T), C, K, dtype, act=("silu", "none")[K % 2], state=C % 3 != 0,
               final=C % 2 == 0, bias=K != 3, pdt=("f32", dtype)[K % 2])


@pytest.mark.parametrize("T", [1, 2, 3, 4, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 513])
@pytest.mark.parametrize("C", [5, 256])
def test_causal_conv_lengths(C, T):
    check_conv(np.random.default_rng(T), (2, T), C, 4, "f32")


PACKED = [[0, 5, 5, 6, 40, 41], [0, 0, 3], [3, 3, 90, 90, 100], [2, 2], [0, 300], [7, 8, 9, 10, 12, 15, 19, 64, 128, 131]]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offsets", PACKED)
@pytest.mark.parametrize("C,K", [(16, 4), (7, 3), (40, 6)])
def test_causal_conv_packed(C, K, offsets, dtype):
    check_conv(np.random.default_rng(len(offsets)), (offsets[-1] + 4,), C, K, dtype, offsets=offsets, state=C != 7)


def strided(dtype, pad, order=None):
    """Views into larger tensors: `pad` extra channels on either side, or positions before sequences."""
    rng = np.random.default_rng(3)

    def make(shape):
        if order == "time first":
            return rand(rng, (shape[1], shape[0], shape[2] + pad), dtype).transpose(0, 1)[..., pad:]
        if order == "every second":
            return rand(rng, (shape[0], 2 * shape[1], shape[2] + pad), dtype)[:, ::2, pad:]
        return rand(rng, (*shape[:-1], shape[-1] + 2 * pad), dtype)[..., pad:-pad]
    return make


@pytest.mark.parametrize("pad,order", [(8, None), (3, None), (8, "time first"), (1, "every second"), (16, "every second")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_causal_conv_views(dtype, pad, order):
    check_conv(np.random.default_rng(1), (3, 40), 32, 4, dtype, view=strided(dtype, pad, order))


def test_causal_conv_of_a_repeated_row():
    """Inputs broadcast along positions (stride 0)."""
    check_conv(np.random.default_rng(1), (2, 20), 16, 3, "f32",
               view=lambda s: torch.randn(2, 1, 16, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).expand(s))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("C,K,B", [(1, 1, 1), (16, 4, 5), (33, 3, 2), (264, 16, 3), (4096, 4, 64)])
def test_causal_conv_step(B, K, C, dtype):
    """Token by token: the same values as the whole sequence, state in place, a slice of a larger cache."""
    rng = np.random.default_rng(B)
    T = 6
    x, w, b = rand(rng, (B, T, C), dtype), rand(rng, (K, C), "f32", 0.7), rand(rng, C, "f32")
    cache = rand(rng, (B, 2, K - 1, C), dtype)
    start = cache.clone()
    state = cache[:, 1]
    ys = torch.stack([dwc.causal_conv_step(x[:, t], state, w, b, "silu") for t in range(T)], 1)
    want = [ref.causal_conv(d(x[i]), d(w), d(b), "silu", d(start[i, 1])) for i in range(B)]
    within(ys, ref.stack([f[0] for f in want]), "y")
    assert torch.equal(state, torch.from_numpy(np.stack([f[1] for f in want])).to(state.dtype).cuda())
    assert torch.equal(cache[:, 0], start[:, 0])


# ------------------------------------------------------------------------- selective scan

def scan_inputs(rng, lead, C, N, G, dtype, gate=True, skip=True, bias=True, plus=True, view=None):
    make = view or (lambda shape: rand(rng, shape, dtype))
    s = {"u": make((*lead, C)), "dt": make((*lead, C)), "B": rand(rng, (*lead, G, N), dtype), "C": rand(rng, (*lead, G, N), dtype)}
    if not plus:
        s["dt"] = s["dt"].abs() * 0.1
    s["z"] = make((*lead, C)) if gate else None
    s["A"] = -torch.exp(rand(rng, (C, N), "f32", 0.7))
    s["D"] = rand(rng, C, "f32") if skip else None
    s["dt_bias"] = rand(rng, C, "f32", 1.0, -2.0) if bias else None
    return s


def want_scan(s, dy, plus, offsets, count, state, dfinal):
    C, N = s["A"].shape
    zero, none = np.zeros((C, N)), np.zeros(C)
    rows = {k: pieces(s[k], offsets) for k in ("u", "dt", "z", "B", "C") if s[k] is not None}
    dys = pieces(dy, offsets)
    fwd, bwd = [], []
    for i in range(count):
        args = (rows["u"][i], rows["dt"][i], d(s["A"]), rows["B"][i], rows["C"][i], d(s["D"]) if s["D"] is not None else none,
                rows["z"][i] if s["z"] is not None else None, d(s["dt_bias"]) if s["dt_bias"] is not None else none, plus,
                d(state[i]) if state is not None else zero)
        fwd.append(ref.scan(*args))
        bwd.append(ref.scan_bwd(dys[i], *args, d(dfinal[i]) if dfinal is not None else zero, None))
    return fwd, bwd


def check_scan(rng, lead, C, N, G, dtype, offsets=None, state=True, dfinal=True, plus=True, **kw):
    count = lead[0] if offsets is None else len(offsets) - 1
    s = scan_inputs(rng, lead, C, N, G, dtype, plus=plus, **kw)
    dy = kw["view"]((*lead, C)) if kw.get("view") else rand(rng, (*lead, C), dtype)
    h0 = rand(rng, (count, C, N), "f32") if state else None
    df = rand(rng, (count, C, N), "f32") if dfinal else None
    off = device(offsets)
    args = [s[k] for k in ("u", "dt", "A", "B", "C")]
    rest = [s[k] for k in ("D", "z", "dt_bias")]
    y, last, saved = dwc.selective_scan_fwd(*args, *rest, plus, h0, off, final=True, save=True)
    got = dwc.selective_scan_bwd(dy, *args, saved, *rest, plus, off, df, state_grad=state)
    got = dict(zip(("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dstate"), got))
    fwd, bwd = want_scan(s, dy, plus, offsets, count, h0, df)
    within(inside(y, offsets), joined([f[0] for f in fwd], offsets), "y")
    within(last, ref.stack([f[1] for f in fwd]), "final")
    for k in ("du", "ddt", "dz", "dB", "dC"):
        if k == "dz" and s["z"] is None:
            assert got[k] is None
            continue
        assert got[k].dtype == DT[dtype]
        within(inside(got[k], offsets), joined([f[k] for f in bwd], offsets), k)
        if offsets is not None:
            assert not got[k][:offsets[0]].any() and not got[k][offsets[-1]:].any()
    within(got["dA"], added([f["dA"] for f in bwd]), "dA")
    for k, given in (("dD", s["D"]), ("ddt_bias", s["dt_bias"])):
        assert (got[k] is None) == (given is None)
        if given is not None:
            within(got[k], added([f[k] for f in bwd]), k)
    if state:
        within(got["dstate"], ref.stack([f["dstate"] for f in bwd]), "dstate")
    else:
        assert got["dstate"] is None
    # a forward pass that keeps less, an output of the caller's, and the same again
    out = torch.full_like(y, 7.0)
    assert dwc.selective_scan_fwd(*args, *rest, plus, h0, off, out=out) is out
    assert torch.equal(inside(out, offsets), inside(y, offsets))
    if offsets is not None:
        assert (out[:offsets[0]] == 7).all() and (out[offsets[-1]:] == 7).all()
    again = dwc.selective_scan_bwd(dy, *args, saved, *rest, plus, off, df, state_grad=state)
    assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(again, got.values()))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("N", [1, 2, 4, 7, 8, 11, 12, 16, 17, 24, 32, 33, 40, 64, 65, 72, 100, 128])
def test_scan_states(N, dtype):
    rng = np.random.default_rng(N)
    check_scan(rng, (2, 37), 19 if N % 2 else 40, N, 1, dtype, gate=N % 3 != 0, state=N % 4 != 0, dfinal=N % 4 != 1)


@pytest.mark.parametrize("T", [1, 2, 3, 8, 31, 32, 33, 63, 64, 65, 96, 130])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_lengths(T, dtype):
    check_scan(np.random.default_rng(T), (2, T), 24, 16, 1, dtype)


@pytest.mark.parametrize("C,G", [(1, 1), (6, 6), (12, 3), (64, 4), (70, 2), (96, 1), (130, 1)])
@pytest.mark.parametrize("N", [5, 16])
def test_scan_channels_and_groups(C, G, N):
    check_scan(np.random.default_rng(C), (3, 20), C, N, G, "f32")


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("skip,bias,plus", [(True, True, True), (False, True, True), (True, False, True), (False, False, False)])
def test_scan_options(gate, skip, bias, plus):
    check_scan(np.random.default_rng(2), (2, 21), 16, 8, 2, "f32", gate=gate, skip=skip, bias=bias, plus=plus, state=gate,
               dfinal=skip)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offsets", PACKED)
@pytest.mark.parametrize("C,N,G", [(16, 16, 1), (7, 3, 1), (40, 24, 2)])
def test_scan_packed(C, N, G, offsets, dtype):
    check_scan(np.random.default_rng(len(offsets)), (offsets[-1] + 5,), C, N, G, dtype, offsets=offsets, state=C != 7)


@pytest.mark.parametrize("pad,order", [(8, None), (3, None), (8, "time first"), (1, "every second")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_views(dtype, pad, order):
    check_scan(np.random.default_rng(1), (3, 34), 32, 16, 1, dtype, view=strided(dtype, pad, order))


def test_scan_slices_of_one_projection():
    """dt, B and C as the slices of one matrix, B and C without an axis of groups."""
    rng = np.random.default_rng(4)
    C, N = 24, 10
    x = rand(rng, (2, 33, C + 2 * N + 3), "bf16")
    s = scan_inputs(rng, (2, 33), C, N, 1, "bf16")
    s["dt"], s["B"], s["C"] = x[..., :C], x[..., C:C + N], x[..., C + N + 3:]
    y = dwc.selective_scan_fwd(s["u"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"])
    s["B"], s["C"] = s["B"][:, :, None], s["C"][:, :, None]
    fwd, _ = want_scan(s, s["u"], True, None, 2, None, None)
    within(y, ref.stack([f[0] for f in fwd]), "y")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,C,N,G", [(1, 1, 1, 1), (3, 24, 16, 1), (2, 33, 11, 3), (5, 64, 128, 2), (2, 40, 50, 1), (64, 1024, 16, 1)])
def test_scan_step(B, C, N, G, dtype):
    rng = np.random.default_rng(C)
    T = 4
    s = scan_inputs(rng, (B, T), C, N, G, dtype)
    cache = rand(rng, (B, 2, C, N), "f32")
    start, state = cache.clone(), cache[:, 0]
    ys = torch.stack([dwc.selective_scan_step(s["u"][:, t], s["dt"][:, t], s["A"], s["B"][:, t], s["C"][:, t], state, s["D"],
                                              s["z"][:, t], s["dt_bias"]) for t in range(T)], 1)
    none = np.zeros(C)
    want = [ref.scan(d(s["u"][i]), d(s["dt"][i]), d(s["A"]), d(s["B"][i]), d(s["C"][i]), d(s["D"]), d(s["z"][i]), d(s["dt_bias"]) + none,
                     True, d(start[i, 0])) for i in range(B)]
    within(ys, ref.stack([f[0] for f in want]), "y")
    within(state, ref.stack([f[1] for f in want]), "state")
    assert torch.equal(cache[:, 1], start[:, 1])


def test_scan_forgets_everything_at_large_steps():
    """exp(delta A) underflows to zero: only the last input counts, and its gradients; no NaN."""
    rng = np.random.default_rng(0)
    s = scan_inputs(rng, (2, 40), 16, 8, 1, "f32")
    s["dt"] = s["dt"] * 3 + 300.0
    dy = rand(rng, (2, 40, 16), "f32")
    args, rest = [s[k] for k in ("u", "dt", "A", "B", "C")], [s[k] for k in ("D", "z", "dt_bias")]
    y, saved = dwc.selective_scan_fwd(*args, *rest, save=True)
    got = dwc.selective_scan_bwd(dy, *args, saved, *rest)
    fwd, bwd = want_scan(s, dy, True, None, 2, None, None)
    within(y, ref.stack([f[0] for f in fwd]), "y")
    for t, k in zip(got, ("du", "ddt", None, "dB", "dC")):
        assert t.isfinite().all()
        if k:
            within(t, ref.stack([f[k] for f in bwd]), k)


def test_a_bad_channel_or_sequence_stays_alone():
    """Infinities and NaN of one sequence, of one channel's u, dt or z and of rows beside the sequences reach
    nothing else (B and C are shared by a group's channels, so they are kept finite)."""
    rng = np.random.default_rng(0)
    s = scan_inputs(rng, (80,), 40, 16, 1, "f32")
    off = torch.tensor([4, 30, 70], dtype=torch.int32, device="cuda")
    run = lambda: dwc.selective_scan_fwd(s["u"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"],  # noqa: E731
                                         offsets=off, final=True)
    good, last = run()
    conv = dwc.causal_conv_fwd(s["u"], s["A"][:, :4].t().contiguous(), None, "silu", offsets=off)
    for k in ("u", "dt", "z", "B", "C"):
        s[k][:4] = float("nan")
        s[k][70:] = float("inf")
    s["u"][10, 3], s["dt"][11, 5], s["z"][12, 9] = float("inf"), float("nan"), float("nan")
    bad, last2 = run()
    keep = torch.ones_like(good, dtype=torch.bool)
    keep[4:30, [3, 5, 9]] = False
    assert torch.equal(good[keep], bad[keep]) and bad[4:30, 3].isnan().sum() + bad[4:30, 3].isinf().sum() > 0
    rows = [c for c in range(40) if c not in (3, 5)]
    assert torch.equal(last[1], last2[1]) and torch.equal(last[0, rows], last2[0, rows])
    conv2 = dwc.causal_conv_fwd(s["u"], s["A"][:, :4].t().contiguous(), None, "silu", offsets=off)
    keep[:] = True
    keep[10:14, 3] = False
    assert torch.equal(conv[keep], conv2[keep]) and not conv2[10, 3].isfinite()


# ----------------------------------------------------------------------------- block norm

PAIRS = [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("f32", "f16")]


def check_norm(rng, shape, wide, dtype, act="silu", params=(True, True, True), alpha=0.9, eps=1e-5, dz=True, pdt="f32", view=None,
               inplace=False):
    C = shape[-1]
    make = view or (lambda t: rand(rng, shape, t))
    x, gate, res, dy = make(dtype), make(dtype) if act else None, make(wide), make(dtype)
    dzt = make(wide) if dz else None
    gpost, gpre, scale = (rand(rng, C, pdt, 0.3, 1.0) if p else None for p in params)
    res0 = res.clone()
    y, z, post, pre = dwc.block_norm_fwd(x, res, gpost, gpre, gate, scale, alpha, act or "none", eps, z=res if inplace else None, stats=True)
    flat = lambda t: d(t).reshape(-1, C)  # noqa: E731
    one = np.ones(C)
    p = [d(t) if t is not None else one for t in (gpost, gpre, scale)]
    want = ref.block_norm(flat(x), flat(res0), p[0], p[1], flat(gate) if act else None, p[2], alpha, act, eps)
    for name, got, w in zip(("y", "z", "rstd_post", "rstd_pre"), (y, z, post, pre), want):
        within(got.reshape(w.v.shape), w, name)
    assert y.dtype == DT[dtype] and z.dtype == DT[wide] and (not inplace or z is res)
    y2, z2 = dwc.block_norm_fwd(x, res0, gpost, gpre, gate, scale, alpha, act or "none", eps)
    assert torch.equal(y, y2) and torch.equal(z, z2)
    got = dwc.block_norm_bwd(dy, x, z, post, pre, gpost, gpre, gate, scale, alpha, act or "none", dzt)
    want = ref.block_norm_bwd(flat(dy), flat(x), flat(z), d(post).reshape(-1), d(pre).reshape(-1), p[0], p[1], flat(gate) if act else None,
                              p[2], alpha, act or "none", flat(dzt) if dz else np.zeros_like(flat(x)))
    has = {"dgate": bool(act), "dgamma_post": params[0], "dgamma_pre": params[1], "dscale": params[2]}
    for name, g in zip(("dx", "dres", "dgate", "dgamma_post", "dgamma_pre", "dscale"), got):
        assert (g is not None) == has.get(name, True), name
        if g is not None:
            within(g.reshape(want[name].v.shape), want[name], name)
    only = dwc.block_norm_bwd(dy, x, z, post, pre, gpost, gpre, gate, scale, alpha, act or "none", dzt, param_grads=False)
    assert only[3:] == (None, None, None) and torch.equal(only[0], got[0]) and torch.equal(only[1], got[1])


CHANNELS = [1, 2, 7, 8, 9, 31, 32, 64, 65, 96, 100, 127, 128, 129, 250, 256, 257, 512, 513, 1000, 1001, 1024, 1025, 2048, 2056, 4096, 4099,
            5000, 8192, 8200, 16384, 20001]


@pytest.mark.parametrize("pair", PAIRS, ids="-".join)
@pytest.mark.parametrize("C", CHANNELS)
def test_block_norm(C, pair):
    rows = {0: 1, 1: 37, 2: 130}[C % 3] if C < 5000 else 5
    check_norm(np.random.default_rng(C), (rows, C), *pair, act=("silu", "sigmoid", None, "none")[C % 4], dz=C % 5 != 0,
               inplace=C % 2 == 0)


@pytest.mark.parametrize("rows", [1, 2, 3, 8, 9, 151, 152, 153, 305, 609, 1300])
@pytest.mark.parametrize("C", [72, 1001, 2048])
def test_block_norm_row_counts(rows, C):
    check_norm(np.random.default_rng(rows), (rows, C), "f32", "bf16")


@pytest.mark.parametrize("params", [(True, False, False), (False, True, False), (False, False, True), (False, False, False)])
@pytest.mark.parametrize("pdt", DT)
@pytest.mark.parametrize("C", [100, 2048])
def test_block_norm_parameters(C, pdt, params):
    check_norm(np.random.default_rng(4), (19, C), "bf16", "bf16", params=params, pdt=pdt, alpha=1.0)


@pytest.mark.parametrize("pair", PAIRS, ids="-".join)
@pytest.mark.parametrize("view", [
    lambda rng, t: rand(rng, (40, 300), t)[:, 16:272], lambda rng, t: rand(rng, (40, 300), t)[:, 5:205],
    lambda rng, t: rand(rng, (40, 2056), t)[:, 1:2050], lambda rng, t: rand(rng, (33, 128), t)[::3],
    lambda rng, t: rand(rng, (33, 129), t)[1:], lambda rng, t: rand(rng, (3, 5, 7, 96), t)])
def test_block_norm_views(view, pair):
    rng = np.random.default_rng(5)
    check_norm(rng, tuple(view(rng, "f32").shape), *pair, view=lambda t: view(rng, t))


def test_block_norm_of_zero_rows_and_zero_values():
    x = torch.zeros(3, 64, device="cuda")
    y, z, post, pre = dwc.block_norm_fwd(x, x.clone(), eps=1e-6, stats=True)
    assert not y.any() and not z.any() and torch.allclose(post, torch.full_like(post, 1e3))
    none = x[:0]
    y, z = dwc.block_norm_fwd(none, none.clone())
    assert y.shape == none.shape
    g = dwc.block_norm_bwd(none, none, none, post[:0], pre[:0], x[0], x[0], None, x[0])
    assert g[0].shape == none.shape and not g[3].any() and not g[4].any() and not g[5].any()


# ------------------------------------------------------------------- a run of them together

def block(p, x, res, state=None):
    """One state space block and the norms around it; x is the normed input."""
    h = x @ p["w_in"]
    C = p["A"].shape[0]
    c = dwc.causal_conv_fwd(h[..., :C], p["w"], p["bias"], "silu", final=True)
    s = c[0] @ p["w_x"]
    N = p["A"].shape[1]
    y = dwc.selective_scan_fwd(c[0], s[..., :C], p["A"], s[..., C:C + N], s[..., C + N:], p["D"], h[..., C:], p["dt_bias"], final=True)
    out, z = dwc.block_norm_fwd(y[0] @ p["w_out"], res, p["g0"], p["g1"], None, p["scale"])
    return out, z, c[1], y[1]


def block_step(p, x, res, conv, state):
    C, N = p["A"].shape
    h = x @ p["w_in"]
    c = dwc.causal_conv_step(h[:, :C], conv, p["w"], p["bias"], "silu")
    s = c @ p["w_x"]
    y = dwc.selective_scan_step(c, s[:, :C], p["A"], s[:, C:C + N], s[:, C + N:], state, p["D"], h[:, C:], p["dt_bias"])
    return dwc.block_norm_fwd(y @ p["w_out"], res, p["g0"], p["g1"], None, p["scale"])


def block_params(W, C, N, K, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return {"w_in": r(W, 2 * C) / W ** 0.5, "w": r(K, C) / 2, "bias": 0.1 * r(C), "w_x": r(C, C + 2 * N) / C ** 0.5, "A": -torch.exp(r(C, N)),
            "D": r(C), "dt_bias": r(C) - 2, "w_out": r(C, W) / C ** 0.5, "g0": 1 + 0.1 * r(W), "g1": 1 + 0.1 * r(W), "scale": 0.3 + 0.1 * r(W)}


def test_a_prompt_and_its_tokens_are_the_whole_sequence():
    """Prompt by the sequence kernels, then tokens one by one, against one pass over both; replayed from a graph too."""
    W, C, N, K, B, T, more = 48, 64, 16, 4, 3, 41, 5
    p = block_params(W, C, N, K)
    g = torch.Generator("cuda").manual_seed(1)
    x, res = (torch.randn(B, T + more, W, device="cuda", generator=g) for _ in range(2))
    whole, z, conv_end, state_end = block(p, x, res)
    part, _, conv, state = block(p, x[:, :T].contiguous(), res[:, :T].contiguous())
    # fp32 throughout: matrix products of up to 2 C = 128 terms of order 1, in another order: 128 * 2^-24 = 8e-6 relative to their
    # terms, through three products, a scan and a norm: 1e-4 leaves an order of magnitude
    assert torch.allclose(part, whole[:, :T], rtol=1e-4, atol=1e-4)
    xt, rt = torch.empty(B, W, device="cuda"), torch.empty(B, W, device="cuda")
    conv2, state2 = conv.clone(), state.clone()
    ys = []
    for t in range(T, T + more):
        ys.append(block_step(p, x[:, t], res[:, t], conv, state)[0])
        assert torch.allclose(ys[-1], whole[:, t], rtol=1e-4, atol=1e-4)
    assert torch.allclose(state, state_end, rtol=1e-4, atol=1e-4) and torch.allclose(conv, conv_end, rtol=1e-4, atol=1e-4)
    xt.copy_(x[:, T])
    rt.copy_(res[:, T])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block_step(p, xt, rt, conv2.clone(), state2.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = block_step(p, xt, rt, conv2, state2)
    for i, t in enumerate(range(T, T + more)):
        xt.copy_(x[:, t])
        rt.copy_(res[:, t])
        graph.replay()
        assert torch.equal(out, ys[i])
    assert torch.equal(state, state2) and torch.equal(conv, conv2)


def test_two_threads_at_once():
    """Two host threads on streams of their own: the bits of one after the other."""
    rng = np.random.default_rng(8)
    s = scan_inputs(rng, (2, 200), 48, 8, 1, "f32")
    args, rest = [s[k] for k in ("u", "dt", "A", "B", "C")], [s[k] for k in ("D", "z", "dt_bias")]
    w, g = rand(rng, (4, 48), "f32"), rand(rng, 48, "f32")

    def passes():
        y, saved = dwc.selective_scan_fwd(*args, *rest, save=True)
        out = list(dwc.selective_scan_bwd(y, *args, saved, *rest)[:8])
        out += [dwc.causal_conv_fwd(y, w, g), *dwc.causal_conv_bwd(y, s["u"], w, g, "silu")[:3]]
        n, z, post, pre = dwc.block_norm_fwd(y, s["u"], g, g, s["z"], g, stats=True)
        return [y, n, z, *out, *dwc.block_norm_bwd(n, y, z, post, pre, g, g, s["z"], g)]

    want = passes()
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i] = passes()
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for side in got:
        assert len(side) == len(want) and all(torch.equal(a, b) for a, b in zip(side, want))


def test_streams_and_graphs_of_the_training_passes():
    """On another stream, and captured: the same bits as eager calls; two graphs that replay in turn keep their own workspaces."""
    rng = np.random.default_rng(3)
    s = scan_inputs(rng, (2, 100), 64, 16, 1, "bf16")
    dy = rand(rng, (2, 100, 64), "bf16")
    w, b = rand(rng, (4, 64), "f32"), rand(rng, 64, "f32")
    args, rest = [s[k] for k in ("u", "dt", "A", "B", "C")], [s[k] for k in ("D", "z", "dt_bias")]

    def step(stream=None):
        y, saved = dwc.selective_scan_fwd(*args, *rest, save=True, stream=stream)
        g = dwc.selective_scan_bwd(dy, *args, saved, *rest, stream=stream)
        c = dwc.causal_conv_bwd(dy, s["u"], w, b, "silu", stream=stream)
        n = dwc.block_norm_fwd(y, s["u"], b, b, s["z"], b, stats=True, stream=stream)
        m = dwc.block_norm_bwd(dy, y, n[1], n[2], n[3], b, b, s["z"], b, stream=stream)
        return [t for t in (y, *g, *c, *n, *m) if t is not None]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        graphs.append((graph, outs))
    for graph, outs in graphs + graphs[::-1]:
        for t in outs:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_binding_refusals():
    x = torch.zeros(2, 3, 8, device="cuda")
    w, st = torch.zeros(4, 8, device="cuda"), torch.zeros(2, 3, 8, device="cuda")
    A, B = torch.zeros(8, 4, device="cuda"), torch.zeros(2, 3, 4, device="cuda")
    off = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    bad = [
        (dwc.causal_conv_fwd, (x[0], w), {}), (dwc.causal_conv_fwd, (x, w[:, :4]), {}), (dwc.causal_conv_fwd, (x, w.t()), {}),
        (dwc.causal_conv_fwd, (x, w, w[0, :4]), {}), (dwc.causal_conv_fwd, (x, w, w[0].half()), {}),
        (dwc.causal_conv_fwd, (x, w, None, "relu"), {}), (dwc.causal_conv_fwd, (x, w, None, "sigmoid"), {}),
        (dwc.causal_conv_fwd, (x, w, None, "none", st[:, :2]), {}), (dwc.causal_conv_fwd, (x, w, None, "none", st.half()), {}),
        (dwc.causal_conv_fwd, (x, w, None, "none", None, off), {}), (dwc.causal_conv_fwd, (x[0], w, None, "none", None, off.long()), {}),
        (dwc.causal_conv_fwd, (x, w), {"out": x}), (dwc.causal_conv_fwd, (x.transpose(1, 2), w), {}),
        (dwc.causal_conv_fwd, (x, w), {"out": torch.zeros(2, 3, 8, device="cuda", dtype=torch.half)}),
        (dwc.causal_conv_bwd, (x[:, :2], x, w), {}), (dwc.causal_conv_bwd, (x.half(), x, w), {}),
        (dwc.causal_conv_step, (x[:, 0], st[:, :2], w), {}), (dwc.causal_conv_step, (x, st, w), {}),
        (dwc.causal_conv_step, (st[:, 0], st, w), {}), (dwc.causal_conv_step, (x[:, 0], st.expand(2, 3, 8)[:1].expand(2, 3, 8), w), {}),
        (dwc.selective_scan_fwd, (x, x[:, :2], A, B, B), {}), (dwc.selective_scan_fwd, (x, x, A.half(), B, B), {}),
        (dwc.selective_scan_fwd, (x, x, A, B[:, :2], B), {}), (dwc.selective_scan_fwd, (x, x, A, B[..., :3], B), {}),
        (dwc.selective_scan_fwd, (x, x, A, B.half(), B), {}), (dwc.selective_scan_fwd, (x, x, A, B, B, A[:, 0]), {}),
        (dwc.selective_scan_fwd, (x, x, A, torch.zeros(2, 3, 3, 4, device="cuda"), torch.zeros(2, 3, 3, 4, device="cuda")), {}),
        (dwc.selective_scan_fwd, (x, x, A, B, B), {"state": A}), (dwc.selective_scan_fwd, (x, x, A, B, B), {"out": x}),
        (dwc.selective_scan_bwd, (x, x, x, A, B, B, A), {}),
        (dwc.selective_scan_step, (x[:, 0], x[:, 0], A, B[:, 0], B[:, 0], A), {}),
        (dwc.block_norm_fwd, (x, x[:1]), {}), (dwc.block_norm_fwd, (x, x.half()), {}), (dwc.block_norm_fwd, (x, x, A[:, 0]), {}),
        (dwc.block_norm_fwd, (x, st, None, None, x.half()), {}), (dwc.block_norm_fwd, (x, st), {"act": "tanh"}),
        (dwc.block_norm_fwd, (x, st), {"out": x.flatten()[:48].view(2, 3, 8)[:, :, :].half()}),
    ]
    for f, args, kw in bad:
        with pytest.raises((ValueError, TypeError, dwc.DwcError)):
            f(*args, **kw)
    torch.cuda.synchronize()
