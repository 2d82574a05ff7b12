"""The conv and scan for single tokens where a block takes several heads: with at least eight blocks an SM (1216 of 152) that way and at most
8192 elements of their states.  Against the fp64 oracle, with its tolerances; padding rows and sequences that begin among the rows."""
import pytest
import torch

from test_conv_scan_step_gpu import BF, F, check, make, ssd  # noqa: F401  (ssd: a fixture)

pytestmark = pytest.mark.gpu

SHAPES = [  # rows, H, P, N, G, K: heads of a block
    (305, 8, 16, 16, 1, 4),     # 2 of 8
    (1300, 8, 16, 16, 1, 4),    # 8
    (700, 12, 33, 20, 2, 3),    # 6, a group's
    (1300, 256, 1, 4, 1, 2),    # 256, more than the block's threads
    (640, 8, 8, 128, 2, 4),     # 4, a group's; whole warps a row
    (640, 4, 24, 64, 1, 4),     # 2 of 4
    (1220, 6, 5, 36, 3, 4),     # 2, a group's
    (1250, 3, 7, 8, 1, 3),      # 3
    (1216, 2, 40, 100, 1, 4),   # 2, the largest states
]


@pytest.mark.parametrize("dtype,ddt", [(BF, BF), (BF, F), (F, F)])
@pytest.mark.parametrize("n,H,P,N,G,K", SHAPES)
def test_several_heads_of_a_block(ssd, n, H, P, N, G, K, dtype, ddt):  # noqa: F811
    s = make(11, n, H, P, N, G, K, dtype, ddt)
    s["slots"][3::17], s["slots"][5::41], s["pos"][7::29] = -1, n + 3, -4
    fresh = s["slots"][11::13][s["slots"][11::13].clamp(0, n + 2) == s["slots"][11::13]].long()
    s["pos"][11::13] = 0
    s["states"][fresh] = 1e30   # (neither the state nor the ring is read at position 0)
    s["ring"][fresh, 1:] = 1e30
    y = check(ssd, s, G)
    assert not y[3::17].any() and not y[5::41].any()
