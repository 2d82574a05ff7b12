"""Infinities and NaN among the values that every row of a tile sees: they give
what the sum gives, p inf = inf for a weight p > 0, inf - inf and NaN not a
number, in the elements that hold them and in no other."""
import numpy as np
import pytest
import torch

from oracle.attention import paged_attention
from test_paged_attn_gpu import BF, C, F, ROUND, make, run, ssd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("lens,new,H,hk,D,ps", [
    ([1, 3], [1, 1], 2, 1, 64, 16),            # a single token: its weight is 1
    ([40, 300], [1, 1], 8, 2, 128, 16),
    ([70, 500], [5, 3], 4, 1, 64, 16),
    ([70, 500], [5, 3], 16, 2, 128, 24),
    ([70, 90], [3, 1], 6, 2, 80, 7),
    ([333, 64], [2, 1], 5, 1, 256, 32),
    ([30, 9, 45, 60] * 50, [1] * 200, 8, 4, 64, 16),
    ([30, 9, 45, 60] * 50, [5] * 200, 8, 2, 128, 16),
])
def test_values_that_every_row_sees(ssd, dtype, lens, new, H, hk, D, ps):
    c = make(51, lens, new, H, hk, D, ps, dtype)
    inf = float("inf")
    for r in range(len(lens)):
        t = 1 if lens[r] - new[r] > 1 else 0   # (a token that the request's first row sees)
        v = c["vc"][int(c["table"][r, t // ps]), t % ps]
        v[:, 3], v[:, D // 2], v[:, D - 1] = inf, -inf, float("nan")
        if t == 1:
            v[:, 10] = inf
            c["vc"][int(c["table"][r, 0]), 0, :, 10] = -inf
    out, lse = run(ssd, c)
    with np.errstate(invalid="ignore"):
        ref, rlse, size = paged_attention(c["q"], c["kc"], c["vc"], c["table"], c["pos"], c["start"], D ** -0.5, 0)
    got = out.double().cpu().numpy()
    assert np.isposinf(ref[..., 3]).all() and np.isneginf(ref[..., D // 2]).all() and np.isnan(ref[..., D - 1]).all()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(np.isposinf(got), np.isposinf(ref)) and np.array_equal(np.isneginf(got), np.isneginf(ref))
    fin = np.isfinite(ref)
    assert (np.abs(got[fin] - ref[fin]) <= ROUND[dtype] * np.abs(ref[fin]) + C * size[fin]).all()
    assert (np.abs(lse.double().cpu().numpy() - rlse) <= C + 2.0 ** -22 * np.abs(rlse)).all()
