"""Updates in place of the norm and dropout operators: an output that is one of the call's inputs gives the
bits of an output of its own, on every kernel; any other overlap is refused.

Parameter gradients of calls of few rows are added up in another order in place (the header says so); they
are held to the bounds of oracle/norm.py against 64 bits."""
import numpy as np
import pytest
import torch

import depthwise_convolution_nhwc_gb300 as dwc
from oracle import norm as ref
from test_norm_gpu import DT, EPS, PAIRS, d, inputs, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dwc.build()
    dwc.load_library()
    yield
    assert dwc.device_status() == 0, "a kernel reported a timed-out wait"


def same(a, b):
    return torch.equal(a.nan_to_num(), b.nan_to_num()) and torch.equal(a.isnan(), b.isnan())


# few rows (one CTA, columns added up in the row kernel) and many; lane groups, one and several groups to a CTA,
# clusters, the general kernels (beyond 65536 channels); aligned and shifted rows
SIZES = [(1, 33), (64, 1000), (200, 4096), (300, 129), (37, 1001), (257, 2048), (640, 5003), (100, 12289), (40, 12288),
         (3, 70001), (2000, 33), (1500, 250)]


@pytest.mark.parametrize("pair", PAIRS, ids="-".join)
@pytest.mark.parametrize("rows,C", SIZES)
def test_backward(rows, C, pair):
    """dx over dy (one type) and over x."""
    s = inputs(rows, C, *pair, seed=rows + C)
    _, mean, rstd = dwc.layer_norm_fwd(s["z"], s["gamma"], s["beta"], EPS, out_dtype=DT[pair[1]], stats=True)
    want = dwc.layer_norm_bwd(s["dy"], s["z"], mean, rstd, s["gamma"])
    m, r, g = d(mean), d(rstd), d(s["gamma"])
    exact = ref.layer_norm_bwd(d(s["dy"]), d(s["z"]), m, r, g)
    bound = ref.layer_norm_bwd_bound(d(s["dy"]), d(s["z"]), m, r, g, pair[0])
    for name in ("dy", "z") if pair[0] == pair[1] else ("z",):
        t = dict(s, **{name: s[name].clone()})
        dx, dgamma, dbeta = dwc.layer_norm_bwd(t["dy"], t["z"], mean, rstd, s["gamma"], out=t[name])
        assert dx is t[name] or dx.data_ptr() == t[name].data_ptr()
        assert same(dx, want[0]), name
        within(dgamma, exact[1], bound[1], f"dgamma, dx over {name}")
        within(dbeta, exact[2], bound[2], f"dbeta, dx over {name}")


@pytest.mark.parametrize("pair", PAIRS, ids="-".join)
@pytest.mark.parametrize("rows,C", SIZES)
def test_forward(rows, C, pair):
    s = inputs(rows, C, *pair, seed=rows + C)
    if pair[0] == pair[1]:
        want = dwc.layer_norm_fwd(s["z"], s["gamma"], s["beta"], EPS, stats=True)
        x = s["z"].clone()
        got = dwc.layer_norm_fwd(x, s["gamma"], s["beta"], EPS, out=x, stats=True)
        assert all(same(a, b) for a, b in zip(got, want)) and same(x, want[0])
    want = dwc.add_layer_norm_fwd(s["x"], s["z"], s["gamma"], s["beta"], EPS, 0.3, 5, 1, stats=True)
    forms = [("x", "res"), ("x", None), (None, "res")]
    if pair[0] == pair[1]:
        forms += [("res", "x"), ("res", None), (None, "x")]
    for out, z in forms:
        t = {"x": s["x"].clone(), "res": s["z"].clone(), None: None}
        got = dwc.add_layer_norm_fwd(t["x"], t["res"], s["gamma"], s["beta"], EPS, 0.3, 5, 1, out=t[out], z=t[z], stats=True)
        assert all(same(a, b) for a, b in zip(got, want)), (out, z)
        assert out is None or same(t[out], want[0])
        assert z is None or same(t[z], want[1])


def test_dropout():
    for rows, C in ((7, 8), (33, 129), (100, 1000)):
        for dt in DT.values():
            x = torch.randn(rows, C, device="cuda").to(dt)
            want = dwc.dropout_fwd(x, 0.4, 3)
            y = x.clone()
            assert same(dwc.dropout_fwd(y, 0.4, 3, out=y), want) and same(y, want)


def test_other_overlaps_are_refused():
    n = 40 * 64
    buf = torch.randn(4 * n, device="cuda")
    x, shifted = buf[:n].view(40, 64), buf[64:64 + n].view(40, 64)
    half = buf.view(torch.bfloat16)[:n].view(40, 64)                    # the same memory as another type
    wide = buf[:2 * n].view(40, 128)[:, :64]                            # rows 128 apart
    dense = buf[:n].view(40, 64)
    free = buf[2 * n:3 * n].view(40, 64)
    st = torch.ones(40, device="cuda")
    gamma = torch.ones(64, device="cuda")
    before = buf.clone()
    bad = [lambda: dwc.layer_norm_fwd(x, out=shifted), lambda: dwc.layer_norm_fwd(shifted, out=x),
           lambda: dwc.layer_norm_fwd(x, out=half), lambda: dwc.layer_norm_fwd(wide, out=dense),
           lambda: dwc.layer_norm_fwd(x, buf[2 * n:2 * n + 64], out=free), lambda: dwc.layer_norm_fwd(x, None, free[3], out=free),
           lambda: dwc.layer_norm_bwd(x, free, st, st, out=shifted), lambda: dwc.layer_norm_bwd(free, x, st, st, out=shifted),
           lambda: dwc.layer_norm_bwd(wide, free, st, st, out=dense),
           lambda: dwc.layer_norm_bwd(x, x, buf[2 * n:2 * n + 40], st, out=free),
           lambda: dwc.layer_norm_bwd(x, x, st, st, free[0], out=free),
           lambda: dwc.dropout_fwd(x, 0.1, 1, out=shifted), lambda: dwc.dropout_bwd(wide, 0.1, 1, out=dense),
           lambda: dwc.dropout_fwd(x, 0.1, 1, free.view(torch.int64)[0, :1], out=free),
           lambda: dwc.add_layer_norm_fwd(x, free, out=shifted), lambda: dwc.add_layer_norm_fwd(free, x, z=shifted),
           lambda: dwc.add_layer_norm_fwd(x, free, gamma, z=x, out=x), lambda: dwc.add_layer_norm_fwd(x.bfloat16(), free, out=half, z=x),
           lambda: dwc.add_layer_norm_fwd(x, free, out=buf[3 * n:].view(40, 64), z=buf[3 * n - 64:4 * n - 64].view(40, 64))]
    for k, f in enumerate(bad):
        with pytest.raises(ValueError, match="overlaps"):
            f()
    torch.cuda.synchronize()
    assert torch.equal(buf, before)


def test_an_output_between_the_rows_of_an_input_is_no_overlap():
    buf = torch.randn(2 * 4096, device="cuda")
    x = buf.view(2, 4096)[:, :64]
    want = dwc.layer_norm_fwd(x.contiguous())
    for at in (64, 1000, 4096 - 128, 4096 + 64):
        out = buf[at:at + 128].view(2, 64)
        assert torch.equal(dwc.layer_norm_fwd(x, out=out), want), at
    for at in (63, 4096 - 127, 4096 + 63):
        with pytest.raises(ValueError, match="overlaps"):
            dwc.layer_norm_fwd(x, out=buf[at:at + 128].view(2, 64))


def test_dx_over_dy_of_few_rows_against_a_dense_copy_many_times():
    """Calls whose CTAs share the columns of the parameter gradients read dy again after dx is stored."""
    for rows, C in ((32, 1000), (64, 4096), (128, 512), (256, 2048)):
        s = inputs(rows, C, "bf16", "bf16", seed=rows)
        _, mean, rstd = dwc.layer_norm_fwd(s["z"], s["gamma"], stats=True)
        want = np.stack([d(t) for t in ref_grads(s, mean, rstd)])
        for _ in range(20):
            dy = s["dy"].clone()
            _, dgamma, dbeta = dwc.layer_norm_bwd(dy, s["z"], mean, rstd, s["gamma"], out=dy)
            got = np.stack([d(dgamma), d(dbeta)])
            # (fp32 sums of up to 256 terms: far below 1e-4 of the largest)
            assert np.abs(got - want).max() <= 1e-4 * np.abs(want).max(), (rows, C)


def ref_grads(s, mean, rstd):
    xhat = (s["z"].double() - mean.double()[:, None]) * rstd.double()[:, None]
    return (s["dy"].double() * xhat).sum(0), s["dy"].double().sum(0)
