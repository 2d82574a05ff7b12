"""Attention over the paged cache for steps that mix single tokens, drafted ones,
whole prompts, requests that bring nothing and padding rows: more requests than
the short schedule takes, in every variant (rows per tile, head sizes, shares of
warps and of CTAs), against the fp64 oracle.  And fp32 with a bound close to its
own arithmetic."""
import numpy as np
import pytest
import torch

from oracle.attention import paged_attention
from test_paged_attn_gpu import BF, F, check, make, run, ssd  # noqa: F401

pytestmark = pytest.mark.gpu


def mixed(seed, nreq, new_of, longest, prompts=0, prompt=0):
    """Lengths, and how many of their tokens are new, of ``nreq`` requests."""
    rng = np.random.default_rng(seed)
    new = rng.choice(new_of, nreq)
    new[rng.permutation(nreq)[:prompts]] = prompt
    lens = np.maximum(rng.integers(0, longest + 1, nreq), new)
    return lens.tolist(), new.tolist()


def with_padding(c, rows, value=float("nan")):
    q = torch.cat([c["q"], torch.full((rows, *c["q"].shape[1:]), value, dtype=c["q"].dtype)])
    return dict(c, q=q, pos=torch.cat([c["pos"], torch.full((rows,), 3, dtype=torch.int32)]))


def padded_check(ssd, c, rows, **kw):
    out, lse = run(ssd, with_padding(c, rows), **kw)
    n = len(c["pos"])
    assert (out[n:] == 0).all() and torch.isneginf(lse[n:]).all()
    check(out[:n], lse[:n], c, **kw)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("D,ps", [(64, 16), (64, 24), (80, 16), (128, 16), (128, 24), (200, 16), (256, 32)])
@pytest.mark.parametrize("group,hk", [(1, 4), (2, 2), (4, 4), (8, 2), (16, 2), (20, 2)])   # 1 to 32 rows, head blocks
@pytest.mark.parametrize("window", [0, 21])
def test_mixed_requests_shares_of_warps(ssd, dtype, D, ps, group, hk, window):
    lens, new = mixed(D + group, 170, [0, 1, 1, 2, 5], 70)
    c = make(81, lens, new, group * hk, hk, D, ps, dtype)
    padded_check(ssd, c, 13, window=window)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("D,ps", [(64, 16), (80, 24), (128, 16), (256, 16)])
@pytest.mark.parametrize("group", [1, 4, 8, 20])
def test_mixed_requests_shares_of_ctas(ssd, dtype, D, ps, group):
    # one key head: fewer tiles than the GPU has warps, but more requests than the short schedule takes
    lens, new = mixed(D + group, 140, [0, 0, 1, 2], 90)
    c = make(82, lens, new, group, 1, D, ps, dtype)
    padded_check(ssd, c, 5)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("H,hk,D,ps,window", [(8, 2, 128, 16, 0), (8, 8, 64, 16, 40), (16, 1, 64, 24, 0), (6, 2, 80, 16, 33)])
def test_prompts_beside_single_tokens(ssd, dtype, H, hk, D, ps, window):
    lens, new = mixed(83, 150, [0, 1, 1, 1], 120, prompts=4, prompt=150)
    c = make(83, lens, new, H, hk, D, ps, dtype)
    padded_check(ssd, c, 40, window=window)


@pytest.mark.parametrize("dtype", [BF, F])
def test_requests_that_bring_nothing_on_either_side(ssd, dtype):
    for nreq, live in ((600, [300]), (600, [0]), (600, [599]), (600, [0, 599]), (129, [64, 65])):
        new = np.zeros(nreq, dtype=int)
        new[live] = 3
        lens = np.where(new > 0, 700, 0).tolist()
        c = make(84, lens, new.tolist(), 8, 2, 64, 16, dtype)
        padded_check(ssd, c, 9)


@pytest.mark.parametrize("dtype", [BF, F])
def test_many_requests(ssd, dtype):
    lens, new = mixed(85, 3000, [0, 1, 1, 3], 20)
    c = make(85, lens, new, 4, 2, 64, 16, dtype)
    padded_check(ssd, c, 100)


@pytest.mark.parametrize("lens,new,H,hk,D,ps", [
    ([1, 2, 3, 5, 8], None, 4, 2, 64, 16),
    ([60, 11, 300], None, 2, 2, 64, 24),
    ([9, 33], [4, 8], 4, 2, 64, 16),
    ([3, 40, 128], None, 2, 1, 128, 16),
    ([7, 64], [2, 2], 8, 2, 128, 16),
    ([5, 50], None, 3, 1, 256, 16),
    ([4, 9, 16, 30] * 50, [1] * 200, 4, 4, 64, 16),
])
def test_fp32_close_to_its_own_arithmetic(ssd, lens, new, H, hk, D, ps):
    # u = 2^-24.  A score is a sum of D products in chains of at most max(D/8, 16) fused steps, then at most 8 more
    # additions: its error is below (max(D/8, 16) + 8) u S, S the sum of its products' magnitudes, and it moves a weight
    # by twice that at most (the maximum's error enters too).  The exponential's argument is rounded twice (|s2| <= 64:
    # 2^-17), its result to 2^-22; sums of at most 300 weights and weighted values are chains of at most 64: 2^-17 of
    # their size.
    c = make(86, lens, new, H, hk, D, ps, F)
    out, lse = run(ssd, c)
    ref, rlse, size = paged_attention(c["q"], c["kc"], c["vc"], c["table"], c["pos"], c["start"], D ** -0.5, 0)
    k = torch.nan_to_num(c["kc"]).double().abs().reshape(-1, hk, D).repeat_interleave(H // hk, 1)
    S = D ** -0.5 * torch.einsum("rhd,thd->rht", c["q"].double().abs(), k).amax(-1).numpy()
    rel = 2 * (max(D / 8, 16) + 8) * 2.0 ** -24 * S + 2.0 ** -17 + 2.0 ** -22 + 2.0 ** -17
    assert np.median(rel) < 2.0 ** -13
    got = out.double().cpu().numpy()
    assert (np.abs(got - ref) <= 2.0 ** -22 * np.abs(ref) + rel[..., None] * size).all()
    assert (np.abs(lse.double().cpu().numpy() - rlse) <= rel + 2.0 ** -22 * np.abs(rlse)).all()
