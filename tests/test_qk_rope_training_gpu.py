"""The gradients of the q/k norm with rotary position at training sizes: more rows
than the launch's blocks take in one trip, queries and keys sharing the blocks
out, a partial last trip.  Bounds as in test_qk_rope_gpu.py; a weight gradient's
sum is longer here, but each thread's own chain is still some hundreds."""
import numpy as np
import pytest
import torch

from oracle.attention import qk_norm_rope_grad
from test_qk_rope_gpu import BF, F, SUMS, make, near, on_gpu, ssd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,Hq,Hk,D,R,dtype", [
    (6007, 8, 2, 128, 128, BF),
    (6007, 8, 2, 128, 64, F),
    (3001, 5, 5, 64, 64, F),
    (9001, 5, 5, 64, 32, BF),
    (4001, 16, 1, 80, 80, BF),     # few key rows: one block or two for them
    (2003, 3, 6, 256, 64, F),
    (70001, 1, 1, 24, 16, BF),
])
@pytest.mark.parametrize("inter", [False, True])
def test_backward(ssd, T, Hq, Hk, D, R, dtype, inter):
    c = make(T + D, T, Hq, Hk, D, R, dtype)
    g = on_gpu(c, Hq, Hk)
    got = ssd.qk_norm_rope_bwd(g["q"], g["k"], g["qw"], g["kw"], g["cos"], g["sin"], g["pos"], g["dq"], g["dk"], eps=1e-5,
                               interleaved=inter)
    torch.cuda.synchronize()
    for n, x, w in (("q", c["q"], c["qw"]), ("k", c["k"], c["kw"])):
        dx, dw, size, wsize = qk_norm_rope_grad(x, w, c["cos"], c["sin"], c["pos"], c["d" + n], 1e-5, inter)
        near(got["d" + n], dx, size, dtype)
        assert (np.abs(got[f"d{n}_weight"].double().cpu().numpy() - dw) <= SUMS * wsize).all()
