"""8-bit rows at the ends of the numbers' range: v = r t with t = h * weight (* SiLU(z)) formed in fp32.

Tolerances: as at ordinary values (2^-17 of the scale without and 2^-16 with the gate's exponential; values within half a step and
2 * 127 of that), and what products below 2^-126 lose: 2^-150 each, in steps of max|t| / 127 with max|t| >= 2^-126 at
most 127 * 2^-24.
"""
import numpy as np
import pytest
import torch

from oracle import layer_step

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd as mod
    return mod


def normal(seed, *shape, dtype=F):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def call(ssd, mode, x, w):
    """(q, scale, v in fp64, largest |t|, relative tolerance)"""
    if mode == "gate":
        z = normal(9, *x.shape, dtype=x.dtype)
        q, scale = ssd.gated_rmsnorm_q8_fwd(x, z, w, EPS)
        v, h = layer_step.add_rmsnorm(x, w, None, EPS, gate=z)
        t, rel = h * w.double().cpu().numpy() * layer_step.silu(z.double().cpu().numpy()), 2.0 ** -16
    else:
        res = None if mode == "plain" else torch.zeros_like(x)
        q, scale, _ = ssd.add_rmsnorm_q8_fwd(x, w, res, eps=EPS)
        v, h = layer_step.add_rmsnorm(x, w, res, EPS)
        t, rel = h * w.double().cpu().numpy(), 2.0 ** -17
    return q.cpu().numpy(), scale.double().cpu().numpy(), v, np.abs(t).max(1), rel


@pytest.mark.parametrize("mode", ["plain", "residual", "gate"])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("D", [64, 1000, 2560, 5120])
def test_rows_of_small_products(ssd, D, dtype, mode):
    """Rows around 2^-20 to 2^-28 with weights around 2^-98: r is about 1000, products 2^-115 to 2^-125, the values and
    scales well above 2^-126 in all rows that count."""
    x = normal(1, 24, D, dtype=dtype) * (2.0 ** (-20 - torch.arange(24) % 9)).to(dtype).cuda()[:, None]
    w = (1.0 + 0.3 * normal(2, D)) * 2.0 ** -98
    q, scale, v, most, rel = call(ssd, mode, x, w)
    want = layer_step.q8_scale(v)
    # (a row whose maximum is as near to the border as the arithmetic's error may lie on either side)
    counts, zero = (most >= 2.0 ** -126 * 1.0001) & (want >= 2.0 ** -126 * 1.0001), (most < 2.0 ** -126 * 0.9999) | (want < 2.0 ** -126 * 0.9999)
    assert counts.sum() >= 12
    assert (np.abs(scale - want)[counts] <= rel * want[counts]).all()
    assert (np.abs(q - v / want[:, None])[counts] <= 0.5 + 2 * 127 * rel + 127 * 2.0 ** -24).all()
    assert not scale[zero].any() and not q[zero].any()


def test_where_rows_become_zero(ssd):
    """One value a row: t = 2^-126 still counts, 2^-127 does not, whatever r is."""
    x = torch.zeros(3, 64, device="cuda")
    x[0, 5], x[1, 5], x[2, 5] = 2.0 ** -25, 2.0 ** -26, 2.0 ** -27
    q, scale, _ = ssd.add_rmsnorm_q8_fwd(x, torch.full((64,), 2.0 ** -100, device="cuda"), eps=EPS)
    ref, _ = layer_step.add_rmsnorm(x, np.full(64, 2.0 ** -100), None, EPS)
    want = layer_step.q8_scale(ref)
    assert q[:, 5].tolist() == [127, 127, 0] and not q[:, :5].any() and not q[:, 6:].any()
    got = scale.double().cpu().numpy()
    assert (np.abs(got - want)[:2] <= 2.0 ** -17 * want[:2]).all() and got[2] == 0 and want[2] > 2.0 ** -126


def test_products_past_the_range(ssd):
    """A product past fp32's largest number makes the row one that holds an infinity, though r would bring it back; others do not see it."""
    x, w = normal(3, 4, 64), torch.ones(64, device="cuda")
    x[1, 7], w[7] = 1e14, 1e25
    x[2, 7], x[3, 7] = 0.0, 1e13
    q, scale, _ = ssd.add_rmsnorm_q8_fwd(x, w, eps=EPS)
    assert scale[1].isnan() and not q[1].any()
    ref, _ = layer_step.add_rmsnorm(x[[0, 2, 3]], w, None, EPS)
    want, got = layer_step.q8_scale(ref), scale[[0, 2, 3]].double().cpu().numpy()
    assert (np.abs(got - want) <= 2.0 ** -17 * want).all()
    assert q[0, 7].abs() == 127 and q[3, 7] == 127 and q[2].abs().max() == 127
