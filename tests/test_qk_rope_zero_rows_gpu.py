"""Rows of zeros, with and without eps: they stay zero, in the cache too, and have
no part in the gradients where eps is 0 (there is none to speak of)."""
import pytest
import torch

from oracle.attention import qk_norm_rope, qk_norm_rope_grad
from test_qk_rope_gpu import BF, F, SUMS, make, near, on_gpu, ssd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("inter", [False, True])
def test_zero_rows(ssd, dtype, eps, inter):
    T, Hq, Hk, D, R = 23, 4, 2, 80, 32
    c = make(71, T, Hq, Hk, D, R, dtype)
    c["pos"] = torch.arange(T, dtype=torch.int32)
    c["qkv"][5], c["qkv"][9, 1], c["qkv"][11, Hq] = 0, 0, 0
    c["dq"][5], c["dq"][9, 1], c["dk"][5], c["dk"][11, 0] = 0, 0, 0, 0   # (with eps the oracle's gradient is theirs over sqrt(eps))
    g = on_gpu(c, Hq, Hk)
    kc = torch.full((6, 4, Hk, D), 7.0, dtype=dtype, device="cuda")
    vc = kc.clone()
    tab = (g["qw"], g["kw"], g["cos"], g["sin"], g["pos"])
    kw = dict(eps=eps, interleaved=inter)
    qo, ko = ssd.qk_norm_rope_fwd(g["q"], g["k"], *tab, v=g["v"], k_cache=kc, v_cache=vc, slots=torch.arange(T, device="cuda"), **kw)
    got = ssd.qk_norm_rope_bwd(g["q"], g["k"], *tab, g["dq"], g["dk"], **kw)
    torch.cuda.synchronize()
    for y in (qo[5], qo[9, 1], ko[5], ko[11, 0], kc.view(-1, Hk, D)[5], kc.view(-1, Hk, D)[11, 0], got["dq"][5], got["dk"][11, 0]):
        assert (y == 0).all()
    assert torch.equal(kc.view(-1, Hk, D)[:T], ko)
    tiny = 1e-300   # (in place of 0: the oracle's rows of zeros are then 0 as well)
    for n, y, x, w in (("q", qo, c["q"], c["qw"]), ("k", ko, c["k"], c["kw"])):
        near(y, *qk_norm_rope(x, w, c["cos"], c["sin"], c["pos"], eps or tiny, inter), dtype)
        dx, dw, size, wsize = qk_norm_rope_grad(x, w, c["cos"], c["sin"], c["pos"], c["d" + n], eps or tiny, inter)
        near(got["d" + n], dx, size, dtype)
        assert (abs(got[f"d{n}_weight"].double().cpu().numpy() - dw) <= SUMS * wsize).all()
