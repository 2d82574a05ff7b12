"""The residual norm's gradients at the ends of the numbers' range.

Tolerances: as in the tests at ordinary values (one rounding of the result, 2^-18 of the terms' magnitude, 2^-17 for the
weight's gradient's sums), and what squares below 2^-126 lose.  Each of them, and the mean, is off by 2^-150 at most (half
the spacing of subnormal numbers), the root by half of the mean's relative error, so the factor r by 2^-150 / mean(h^2); dx has
r up to three times in a term.
"""
import numpy as np
import pytest
import torch

from oracle import layer_step

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
ROUND = {BF: 2.0 ** -8, F: 2.0 ** -24}


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd as mod
    return mod


def normal(seed, *shape, dtype=F, scale=1.0):
    return (scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


@pytest.mark.parametrize("dtype,rdtype", [(BF, BF), (BF, F), (F, F)])
@pytest.mark.parametrize("D", [64, 264, 1000, 4104, 16384])
@pytest.mark.parametrize("scale", [1e-20, 2.0 ** -65, 2.0 ** -70, 1e12])
def test_gradients_of_tiny_and_large_rows(ssd, scale, D, dtype, rdtype):
    """eps 0: the rows' scale leaves the normalised rows as they are and divides the gradients, which stay finite."""
    n = 9
    h, d, w = normal(1, n, D, dtype=rdtype, scale=scale), normal(2, n, D, dtype=dtype), 1.0 + 0.3 * normal(3, D)
    dx, dw = ssd.add_rmsnorm_bwd(h, w, d, eps=0.0)
    rx, rw, sx, sw = layer_step.add_rmsnorm_grad(h, w, d, None, 0.0)
    lost = 2.0 ** -150 / (h.double().cpu().numpy() ** 2).mean(1).min()
    err = np.abs(dx.double().cpu().numpy() - rx)
    assert (err <= ROUND[rdtype] * np.abs(rx) + (2.0 ** -18 + 3 * lost) * sx + 1e-37).all(), (err / sx).max()
    err = np.abs(dw.double().cpu().numpy() - rw)
    assert (err <= 2.0 ** -24 * np.abs(rw) + (2.0 ** -17 + lost) * sw).all(), (err / sw).max()
