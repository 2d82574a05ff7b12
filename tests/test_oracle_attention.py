"""Independent checks of the attention-layer oracle (CPU): the gradients against
central differences of the forward, the rotation's and the norm's invariants,
paged attention against one dense softmax, and the plan's bookkeeping."""
import numpy as np
import pytest

from oracle.attention import paged_attention, plan_step, qk_norm_rope, qk_norm_rope_grad


def _angles(n, R):
    f = 10000.0 ** (-2.0 * np.arange(R // 2) / max(R, 1))
    a = np.arange(n)[:, None] * f[None, :]
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("D,R,inter", [(16, 16, False), (24, 16, True), (8, 0, False)])
def test_gradients_against_differences(D, R, inter):
    rng = np.random.default_rng(3)
    x, w, dy = rng.standard_normal((3, 2, D)), 1 + 0.1 * rng.standard_normal(D), rng.standard_normal((3, 2, D))
    cos, sin = _angles(9, R)
    pos = np.array([4, -1, 8])
    f = lambda x, w: (qk_norm_rope(x, w, cos, sin, pos, 1e-3, inter)[0] * dy).sum()  # noqa: E731
    dx, dw, _, _ = qk_norm_rope_grad(x, w, cos, sin, pos, dy, 1e-3, inter)
    h = 1e-6
    for at in np.ndindex(*x.shape):
        e = np.zeros_like(x)
        e[at] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    for i in range(D):
        e = np.zeros(D)
        e[i] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-7
    assert (dx[1] == 0).all()


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_keeps_lengths_and_relative_positions(inter):
    rng = np.random.default_rng(4)
    D = 32
    cos, sin = _angles(64, D)
    q, k = rng.standard_normal((1, 1, D)), rng.standard_normal((1, 1, D))
    dots = []
    for p in (0, 20):   # q at p + 7, k at p: the product depends on the distance only
        a, _ = qk_norm_rope(q, None, cos, sin, [p + 7], 0.0, inter)
        b, _ = qk_norm_rope(k, None, cos, sin, [p], 0.0, inter)
        assert abs((a * a).sum() - D) < 1e-12
        dots.append((a * b).sum())
    assert abs(dots[0] - dots[1]) < 1e-12


def test_paged_attention_against_dense():
    rng = np.random.default_rng(5)
    L, ps, D, hk, H = 37, 5, 8, 2, 6
    k, v = rng.standard_normal((L, hk, D)), rng.standard_normal((L, hk, D))
    table = np.array([[6, 2, 9, 0, 3, 1, 8, 5]])
    kc, vc = np.full((10, ps, hk, D), np.nan), np.full((10, ps, hk, D), np.nan)
    for t in range(L):
        kc[table[0, t // ps], t % ps], vc[table[0, t // ps], t % ps] = k[t], v[t]
    q = rng.standard_normal((2, H, D))
    for window in (0, 9):
        out, lse, _ = paged_attention(q, kc, vc, table, [L - 2, L - 1], [0, 2], 0.3, window)
        for i in range(2):
            seen = np.arange(L) <= L - 2 + i
            if window:
                seen &= np.arange(L) > L - 2 + i - window
            for h in range(H):
                s = np.where(seen, 0.3 * k[:, h // 3] @ q[i, h], -np.inf)
                p = np.exp(s) / np.exp(s).sum()
                assert np.allclose(out[i, h], p @ v[:, h // 3], atol=1e-13)
                assert abs(lse[i, h] - np.log(np.exp(s).sum())) < 1e-12


def test_plan_hands_out_each_page_once():
    rng = np.random.default_rng(6)
    cap, ps, n = 50, 4, 6
    ring = rng.permutation(cap).astype(np.int32)
    pos, table, lens = np.array([7, 7 + cap]), np.full((n, 10), -1), np.zeros(n, dtype=int)
    for step in range(60):
        new = rng.integers(-1, 12, n)
        new[lens == 0] = np.maximum(new[lens == 0], 0)
        r = plan_step(lens, new, table, ring, pos, ps, 30)
        table, ring, pos, lens = r["table"], r["ring"], r["ring_pos"], r["lens"]
        held = [table[i, :-(-lens[i] // ps)] for i in range(n)]
        free = ring[np.arange(pos[0], pos[1]) % cap]
        assert sorted(np.concatenate([*held, free])) == list(range(cap))
        assert r["granted"].sum() <= 30 and len(set(r["slots"][r["slots"] >= 0])) == r["granted"].sum()
