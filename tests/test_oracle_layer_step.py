"""Pins of oracle/layer_step.py: finite differences, and the oracles of the conv and the scan over whole sequences."""
import numpy as np
import pytest
import torch

import oracle
from oracle import layer_step
from oracle.neighbors import conv1d_silu, gated_rmsnorm


def test_gradients_by_differences():
    rng = np.random.default_rng(0)
    x, res, w, d, dr = (rng.standard_normal(s) for s in ((5, 16), (5, 16), 16, (5, 16), (5, 16)))

    def loss(x, res, w):
        out, h = layer_step.add_rmsnorm(x, w, res, 1e-3)
        return (out * d).sum() + (h * dr).sum()

    dx, dw, _, _ = layer_step.add_rmsnorm_grad(x + res, w, d, dr, 1e-3)
    for at in [(0, 0), (2, 7), (4, 15)]:
        for k in (0, 1):
            args = [x.copy(), res.copy(), w]
            step = 1e-6
            args[k][at] += step
            up = loss(*args)
            args[k][at] -= 2 * step
            assert abs((up - loss(*args)) / (2 * step) - dx[at]) < 1e-6
    for i in (0, 9):
        wp, wm = w.copy(), w.copy()
        wp[i] += 1e-6
        wm[i] -= 1e-6
        assert abs((loss(x, res, wp) - loss(x, res, wm)) / 2e-6 - dw[i]) < 1e-6


def test_gate_is_the_gated_norm():
    g = torch.Generator().manual_seed(1)
    y, z, w = torch.randn(2, 3, 4, 8, generator=g), torch.randn(2, 3, 4, 8, generator=g), torch.randn(32, generator=g)
    ref = gated_rmsnorm(y=y, z=z, weight=w, eps=1e-6)
    got, _ = layer_step.add_rmsnorm(y.reshape(6, 32), w, None, 1e-6, gate=z.reshape(6, 32))
    assert np.allclose(got, ref.reshape(6, 32), rtol=1e-12, atol=1e-14)


def test_zero_rows():
    out, _ = layer_step.add_rmsnorm(np.zeros((1, 8)), np.ones(8), None, 0.0)
    dx, dw, _, _ = layer_step.add_rmsnorm_grad(np.zeros((1, 8)), np.ones(8), np.ones((1, 8)), None, 0.0)
    assert not out.any() and not dx.any() and not dw.any()


@pytest.mark.parametrize("K,G", [(2, 1), (3, 2), (4, 1)])
def test_steps_are_the_sequence(K, G):
    """Tokens one at a time from position 0 give what the conv's and the scan's oracles give for the sequence."""
    H, P, N, L = 4, 8, 4, 9
    C = H * P + 2 * G * N
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    xbc, w, b, dt, dtb, al, D = r(1, L, C), r(C, K), r(C), r(1, L, H), r(H), r(H), r(H)
    x, B, Cm, _ = conv1d_silu(xbc=xbc, weight=w, bias=b, conv_state=None, H=H, P=P, G=G, N=N)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a))  # noqa: E731
    y, final = oracle.ssd_fwd(x=t(x), dt_raw=dt, dt_bias=dtb, A_log=al, B=t(B), C=t(Cm), D=D, init_state=None)
    ring, states = r(3, K, C), r(3, H, P, N)
    for i in range(L):
        got, ring, states, _ = layer_step.conv_scan_step(xbc[0, i:i + 1], ring, w, b, dt[0, i:i + 1], dtb, al, D, states,
                                                         torch.tensor([1]), torch.tensor([i]), G)
        assert np.allclose(got[0], np.asarray(y)[0, i], rtol=1e-5, atol=1e-6)
    assert np.allclose(states[1], np.asarray(final)[0], rtol=1e-5, atol=1e-6)
