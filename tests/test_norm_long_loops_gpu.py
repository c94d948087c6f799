"""Rows enough that every group of threads works through several rounds, against 64 bits: clusters (their two
exchanges and phases, refilled stages, a live second row, partial gradients over several rows) and the
layouts between 2057 and 4094 channels (one, two and three groups to a CTA, one and two rows at a time).

Row counts leave odd remainders.  A GPU of 152 SMs holds 17 to 76 clusters of 8 to 2 CTAs."""
import pytest
import torch

import depthwise_convolution_nhwc_gb300 as dwc
from test_norm_gpu import PAIRS, check_add, check_ln, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dwc.build()
    dwc.load_library()
    yield
    assert dwc.device_status() == 0, "a kernel reported a timed-out wait"


@pytest.mark.parametrize("pair", PAIRS, ids="-".join)
@pytest.mark.parametrize("rows,C", [(301, 10248), (333, 12289), (301, 12288), (157, 20001), (100, 40000), (64, 65536),
                                    (77, 65533)])
def test_clusters(rows, C, pair):
    s = inputs(rows, C, *pair, seed=rows)
    check_ln(s, *pair)
    check_add(s, *pair, p=0.1, dz=rows % 2 == 1, inplace=rows % 3 == 1)


@pytest.mark.parametrize("pair", PAIRS, ids="-".join)
@pytest.mark.parametrize("rows", [37, 1301])
@pytest.mark.parametrize("C", [2064, 2200, 2561, 2568, 2999, 3000, 3064, 3071, 3080, 3333, 3600, 3999, 4088])
def test_mid_widths(rows, C, pair):
    s = inputs(rows, C, *pair, seed=rows + C)
    check_ln(s, *pair)
    check_add(s, *pair, p=0.1, dz=C % 3 != 0, inplace=C % 2 == 0)


@pytest.mark.parametrize("C", [10248, 12289, 40000])
def test_rows_do_not_depend_on_the_rows_beside_them(C):
    """The rounds a cluster has behind it leave no trace: a call's rows are those of calls of fewer rows from the
    same place (by 8 rows, which keeps a row's shift)."""
    s = inputs(160, C, "bf16", "bf16", seed=C)
    y, mean, rstd = dwc.layer_norm_fwd(s["z"], s["gamma"], s["beta"], stats=True)
    dx = dwc.layer_norm_bwd(s["dy"], s["z"], mean, rstd, s["gamma"])[0]
    for a, b in ((0, 8), (72, 88), (152, 160)):
        y2, m2, r2 = dwc.layer_norm_fwd(s["z"][a:b], s["gamma"], s["beta"], stats=True)
        assert torch.equal(y[a:b], y2) and torch.equal(mean[a:b], m2) and torch.equal(rstd[a:b], r2)
        assert torch.equal(dx[a:b], dwc.layer_norm_bwd(s["dy"][a:b], s["z"][a:b], m2, r2, s["gamma"])[0])
