"""Rows over clusters whose exchange between CTAs does not come: each thread's wait runs out once, the call
ends promptly, the status word says so, and the context stays usable.  No GPU fault is involved: one CTA of
each cluster is told to send its sums to nobody (include/dwc_testing.h)."""
import time

import pytest
import torch

import depthwise_convolution_nhwc_gb300 as dwc
from test_norm_gpu import inputs

pytestmark = pytest.mark.gpu

DWC_OK, DWC_ERR_TIMEOUT = 0, 6


@pytest.mark.parametrize("pair", [("f32", "bf16"), ("bf16", "bf16")], ids="-".join)
@pytest.mark.parametrize("C", [10248, 12289, 65536])
def test_a_lost_exchange_is_reported(C, pair):
    s = inputs(100, C, *pair, seed=C)
    lib = dwc.load_library()
    stats = dwc.layer_norm_fwd(s["z"], stats=True)[1:]

    def forward():
        return dwc.add_layer_norm_fwd(s["x"], s["z"], s["gamma"], s["beta"], p=0.1, seed=3, stats=True)

    def backward():
        return dwc.add_layer_norm_bwd(s["dy"], s["z"], *stats, s["gamma"], s["dz"], 0.1, 3)

    for call in (forward, backward):
        want = call()
        assert dwc.device_status() == DWC_OK
        prev = dwc.set_wait_limit_ns(1_000_000)
        try:
            lib.dwc_testing_stall_next_norm_cluster()
            dwc.layer_norm_fwd(s["z"][:, :4096])      # (no cluster serves it: the request stays)
            t0 = time.perf_counter()
            call()
            status = dwc.device_status()
            elapsed = time.perf_counter() - t0
        finally:
            dwc.set_wait_limit_ns(prev)
        assert status == DWC_ERR_TIMEOUT
        assert elapsed < 1.0, elapsed                 # the limit of 1 ms, not the 2 s default, ended it
        assert dwc.device_status() == DWC_OK          # reading the status cleared it
        again = call()
        assert dwc.device_status() == DWC_OK
        assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_a_limit_shorter_than_any_exchange():
    """1 ns: a wait suspends its thread for longer than that before it looks at the clock, so such calls end well;
    what holds in any case is that a call whose status is clear has the right bits."""
    s = inputs(100, 12289, "bf16", "bf16", seed=1)
    want = dwc.layer_norm_fwd(s["z"], s["gamma"], s["beta"], stats=True)
    prev = dwc.set_wait_limit_ns(1)
    try:
        for _ in range(20):
            got = dwc.layer_norm_fwd(s["z"], s["gamma"], s["beta"], stats=True)
            code = dwc.device_status()
            assert code in (DWC_OK, DWC_ERR_TIMEOUT)
            assert code != DWC_OK or all(torch.equal(a, b) for a, b in zip(got, want))
    finally:
        dwc.set_wait_limit_ns(prev)
