"""Attention over the paged cache at the ends of the positions' range: contexts up
to page_size * max_pages = 2^31 - 2 tokens, and negative positions of any size."""
import numpy as np
import pytest
import torch

from oracle.attention import paged_attention
from test_paged_attn_gpu import BF, F, check, make, run, ssd, to_gpu  # noqa: F401

pytestmark = pytest.mark.gpu

PS, COLS = 331 * 151, 2 * 9 * 7 * 11 * 31   # pages of 49981 tokens, 42966 of them


def far(dtype, D, hk, live, new):
    """One request whose context is as long as a table can make it, with pages in the table's columns ``live`` only, the
    last of them the table's last, and ``new`` query rows; and the same over a table of nothing but those pages."""
    rng = np.random.default_rng(61)
    n = len(live)
    kc, vc = (torch.from_numpy(rng.standard_normal((n, PS, hk, D), dtype=np.float32)).to(dtype) for _ in range(2))
    table = torch.full((1, COLS), -1, dtype=torch.int32)
    table[0, live] = torch.arange(n, dtype=torch.int32)
    q = torch.from_numpy((1.5 * rng.standard_normal((new, 2 * hk, D))).astype(np.float32)).to(dtype)
    pos = PS * COLS - new + np.arange(new)
    start = torch.tensor([0, new], dtype=torch.int32)
    c = dict(q=q, kc=kc, vc=vc, table=table, pos=torch.from_numpy(pos.astype(np.int32)), start=start)
    short = dict(c, table=torch.arange(n, dtype=torch.int32)[None], pos=torch.from_numpy((pos - PS * (COLS - n)).astype(np.int32)))
    return c, short


@pytest.mark.parametrize("dtype,D", [(BF, 8), (BF, 64), (BF, 192), (F, 8), (F, 128)])
@pytest.mark.parametrize("new", [1, 3])
@pytest.mark.parametrize("window", [40, 130])
def test_window_at_the_last_position(ssd, dtype, D, new, window):
    c, short = far(dtype, D, 1, [COLS - 1], new)
    check(*run(ssd, c, window=window), short, window=window)


@pytest.mark.parametrize("dtype,D", [(BF, 64), (F, 8)])
def test_whole_context_up_to_the_last_position(ssd, dtype, D):
    c, short = far(dtype, D, 1, [17, COLS // 2, COLS - 1], 2)
    check(*run(ssd, c), short)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("lowest", [-1, -5, -2 ** 31 + 3, -2 ** 31])
def test_negative_positions_beside_others(ssd, dtype, lowest):
    # two padding rows share a tile with rows of tokens
    c = make(62, [40], [4], 2, 1, 64, 16, dtype)
    c["pos"][:2] = lowest
    check(*run(ssd, c, window=10), c, window=10)
