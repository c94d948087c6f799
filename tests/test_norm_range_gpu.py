"""Rows of very little spread with eps = 0: rstd is near the square root of the largest float, dx is finite,
and every kernel gives it (no square of rstd on the way)."""
import numpy as np
import pytest
import torch

import depthwise_convolution_nhwc_gb300 as dwc
from oracle import norm as ref
from test_norm_gpu import DT, d, within

pytestmark = pytest.mark.gpu

# Spreads down to 2.5e-19: the variance, 6e-38, is a normal fp32 number still.
SPREADS = [3e-18, 2.5e-19]


@pytest.mark.parametrize("pair", [("f32", "f32"), ("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16")], ids="-".join)
@pytest.mark.parametrize("spread", SPREADS)
@pytest.mark.parametrize("rows,C", [(5, 64), (70, 512), (300, 1000), (33, 4096), (9, 8200), (6, 12288), (7, 33), (40, 1001),
                                    (5, 12289), (2, 70001)])
def test_backward_of_rows_with_little_spread(rows, C, spread, pair):
    """dy follows the normalised rows, so that the mean of dy * xhat is near 1 (its sum near C)."""
    wide, narrow = pair
    rng = np.random.default_rng(C)
    hat = rng.standard_normal((rows, C))
    x = torch.from_numpy(hat * spread).to(DT[wide]).cuda()
    dy = torch.from_numpy(hat + 0.5 * rng.standard_normal((rows, C))).to(DT[narrow]).cuda()
    dz = torch.from_numpy(rng.standard_normal((rows, C)) / spread).to(DT[wide]).cuda()
    gamma = torch.from_numpy(1 + 0.2 * rng.standard_normal(C)).float().cuda()
    _, mean, rstd = dwc.layer_norm_fwd(x, gamma, eps=0.0, out_dtype=DT[narrow], stats=True)
    assert torch.isfinite(rstd).all() and float(rstd.min()) > 0.2 / spread
    m, r, g = d(mean), d(rstd), d(gamma)
    got = dwc.layer_norm_bwd(dy, x, mean, rstd, gamma)
    want, bound = ref.layer_norm_bwd(d(dy), d(x), m, r, g), ref.layer_norm_bwd_bound(d(dy), d(x), m, r, g, wide)
    for name, a, w, e in zip(("dx", "dgamma", "dbeta"), got, want, bound):
        within(a, w, e, name)
    dres = dwc.add_layer_norm_bwd(dy, x, mean, rstd, gamma, dz, 0.0)[1]
    within(dres, want[0] + d(dz), ref.layer_norm_bwd_bound(d(dy), d(x), m, r, g, wide, d(dz))[0], "dres")
