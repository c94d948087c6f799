"""Sequence operators where the ordinary inputs of the other tests do not lead: decay rates past fp32's range."""
import numpy as np
import pytest
import torch

import depthwise_convolution_nhwc_gb300 as dwc
from oracle import seq as ref
from test_seq_gpu import added, device, inside, joined, rand, scan_inputs, want_scan, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dwc.build()
    dwc.load_library()
    yield
    assert dwc.device_status() == 0, "a kernel reported a timed-out wait"


def parts(s):
    return [s[k] for k in ("u", "dt", "A", "B", "C")], [s[k] for k in ("D", "z", "dt_bias")]


@pytest.mark.parametrize("rate", [-float("inf"), -3e38])
@pytest.mark.parametrize("lead,C,N,offsets", [((2, 1), 8, 4, None), ((2, 17), 8, 4, None), ((3, 39), 24, 16, None), ((1, 333), 16, 8, None),
                                              ((2, 21), 16, 100, None), ((200,), 12, 5, [0, 3, 20, 36, 199])])
def test_scan_of_states_that_keep_nothing(lead, C, N, offsets, rate):
    """A of minus infinity, and a finite one that log2(e) takes past fp32: exp(delta A) is 0 at every position and its
    derivatives are, as they are of A = -1e6 (delta is 1e-3 and more, exp(-1000) is 0 in 64 bits too)."""
    rng = np.random.default_rng(N)
    count = lead[0] if offsets is None else len(offsets) - 1
    s = scan_inputs(rng, lead, C, N, 1, "f32")
    dy, h0, df = rand(rng, (*lead, C), "f32"), rand(rng, (count, C, N), "f32"), rand(rng, (count, C, N), "f32")
    plain = {**s, "A": s["A"].clone()}
    s["A"][::3, N // 2:], plain["A"][::3, N // 2:] = rate, -1e6
    off = device(offsets)
    args, rest = parts(s)
    y, last, saved = dwc.selective_scan_fwd(*args, *rest, state=h0, offsets=off, final=True, save=True)
    got = dwc.selective_scan_bwd(dy, *args, saved, *rest, offsets=off, dfinal=df, state_grad=True)
    fwd, bwd = want_scan(plain, dy, True, offsets, count, h0, df)
    within(inside(y, offsets), joined([f[0] for f in fwd], offsets), "y")
    within(last, ref.stack([f[1] for f in fwd]), "final")
    for k, t in zip(("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias"), got):
        rows = k in ("du", "ddt", "dB", "dC", "dz")
        within(inside(t, offsets) if rows else t, joined([f[k] for f in bwd], offsets) if rows else added([f[k] for f in bwd]), k)
    within(got[8], ref.stack([f["dstate"] for f in bwd]), "dstate")


def test_scan_step_of_states_that_keep_nothing():
    """A prompt of 16 positions and one token are a prompt of 17."""
    rng = np.random.default_rng(1)
    s = scan_inputs(rng, (3, 17), 24, 8, 1, "f32")
    s["A"][::3, 4:] = -float("inf")
    args, rest = parts(s)
    y, last = dwc.selective_scan_fwd(*args, *rest, final=True)
    cut = lambda t, a, b: t[:, a:b].contiguous()  # noqa: E731
    first, state = dwc.selective_scan_fwd(cut(args[0], 0, 16), cut(args[1], 0, 16), s["A"], cut(args[3], 0, 16), cut(args[4], 0, 16),
                                          rest[0], cut(rest[1], 0, 16), rest[2], final=True)
    one = dwc.selective_scan_step(s["u"][:, 16], s["dt"][:, 16], s["A"], s["B"][:, 16], s["C"][:, 16], state, s["D"], s["z"][:, 16],
                                  s["dt_bias"])
    s["A"][::3, 4:] = -1e6
    fwd, _ = want_scan(s, s["u"], True, None, 3, None, None)
    for got in (y, torch.cat((first, one[:, None]), 1)):
        within(got, ref.stack([f[0] for f in fwd]), "y")
    for got in (last, state):
        within(got, ref.stack([f[1] for f in fwd]), "final")


@pytest.mark.parametrize("T", [37, 300])
def test_scan_of_positions_that_are_left_out(T):
    """delta = 0 leaves the states alone, whatever the (finite) rate."""
    rng = np.random.default_rng(T)
    s = scan_inputs(rng, (2, T), 16, 8, 1, "f32", bias=False, plus=False)
    keep = torch.from_numpy(rng.random((2, T, 1)) < 0.5).cuda()
    s["dt"] = (s["dt"] + 0.01) * keep
    s["A"][:, 4:] = -3e38
    args, rest = parts(s)
    y, last = dwc.selective_scan_fwd(*args, *rest, False, final=True)
    s["A"][:, 4:] = -1e6
    fwd, _ = want_scan(s, s["u"], False, None, 2, None, None)
    within(y, ref.stack([f[0] for f in fwd]), "y")
    within(last, ref.stack([f[1] for f in fwd]), "final")
