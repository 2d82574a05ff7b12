"""Attention over the paged cache where the softmax's exponents are differences of
large scores.  Scores are exact in fp32 here (one or two non-zero elements of
each query row, powers of 2 times numbers of few bits), so whatever error there
is comes from the exponents and the sums, and the bounds are those of
test_paged_attn_gpu.py, which do not grow with the scores."""
import numpy as np
import pytest
import torch

from test_paged_attn_gpu import BF, F, check, make, run, ssd  # noqa: F401

pytestmark = pytest.mark.gpu


def tokens(c, r, n, ps):
    """Pages and offsets of request r's first n tokens."""
    t = np.arange(n)
    return t, torch.from_numpy(c["table"][r].numpy()[t // ps].astype(np.int64)), torch.from_numpy(t % ps)


@pytest.mark.parametrize("dtype", [BF, F])
def test_a_row_whose_maximum_stands_still_among_rows_that_climb(ssd, dtype):
    # More key heads than there are warps, so that a warp takes all units of a tile.  Row 0 of each tile sees equal
    # scores of 512 .. 1020 throughout: its weights are all 1 and lse = score + log n.  The other rows' scores rise past
    # their maximum in every unit, which rescales the tile's rows, row 0 by exactly 1.
    n, hk, D, ps = 1500, 1900, 8, 50
    c = make(41, [n], [4], hk, hk, D, ps, dtype)
    t, page, off = tokens(c, 0, n, ps)
    level = torch.from_numpy((1 + np.arange(hk) % 128 / 128).astype(np.float32)).to(dtype)
    c["kc"][page, off, :, 0] = level[None].expand(n, hk)
    c["kc"][page, off, :, 1] = torch.from_numpy((6.0 * (t // 32)).astype(np.float32)).to(dtype)[:, None].expand(n, hk)
    c["q"][:] = 0
    c["q"][0, :, 0] = 512
    c["q"][1:, :, 1] = 1
    check(*run(ssd, c, scale=1.0), c, scale=1.0)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("lens,new,H,hk,D,ps", [
    ([700], [1], 2, 2, 64, 16),            # one tile in many parts
    ([700, 90], [1, 1], 8, 2, 128, 24),
    ([640, 333], [5, 3], 4, 1, 80, 16),
    ([300, 7, 1], [2, 4, 1], 16, 2, 128, 16),
    ([500, 200], [3, 1], 2, 2, 256, 32),
    ([900, 40, 300, 77] * 40, [1] * 160, 8, 8, 64, 16),   # shares of warps
    ([400, 60] * 30, [1, 1] * 30, 16, 8, 128, 16),
])
@pytest.mark.parametrize("scale", [1.0, -0.7])
def test_scores_past_32_bits(ssd, dtype, lens, new, H, hk, D, ps, scale):
    # scores of 2^33 and more, apart by 2^12 (bf16) or 2^10 (fp32, one unit in the last place) or by 2^26 and more; two
    # tokens share the largest, in different units.  Each row's output is the mean of their values.
    c = make(42, lens, new, H, hk, D, ps, dtype)
    sign = 1.0 if scale > 0 else -1.0
    rng = np.random.default_rng(7)
    step = 2.0 ** 7 if dtype == BF else 2.0 ** 5
    c["q"][:] = 0
    c["q"][:, :, 0], c["q"][:, :, 1] = 2.0 ** 20, 2.0 ** 5
    for r, n in enumerate(lens):
        t, page, off = tokens(c, r, n, ps)
        m = n - new[r] + 1            # tokens that all rows of the request see
        best = rng.permutation(m)[:2]
        top = np.where(rng.random(n) < 0.5, 1.0, rng.integers(64, 127, n) / 128)   # of 2^13, times the head's level
        low = rng.integers(0, 60, n).astype(np.float64)
        top[best], low[best] = 1.0, 63
        level = 1 + np.arange(hk) % 8 / 8   # (with the 7 bits of `top` and those of `low`: at most 24 bits)
        k0 = np.float32(sign * 2.0 ** 13) * torch.from_numpy((top[:, None] * level[None]).astype(np.float32))
        keep = k0.to(torch.bfloat16).to(torch.float32)
        c["kc"][page, off, :, 0] = keep.to(dtype)
        c["kc"][page, off, :, 1] = torch.from_numpy((sign * step * low).astype(np.float32)).to(dtype)[:, None].expand(n, hk)
    check(*run(ssd, c, scale=scale), c, scale=scale)
