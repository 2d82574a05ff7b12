"""GPU parity of the conv and scan for single tokens on a pool of states.

Tolerances: u is a few fp32 operations and an exponential (2^-20 of its terms' magnitude), dt and the decay exponentials
of fp32 numbers (the decay's error grows with |dt A|, and its value falls faster: 2^-19 of the old state), a state two
products and an addition, y a sum of at most 512 terms in 16 sequential additions and a tree: 2^-17 of the magnitude of
the terms; the result's rounding beside it.  What the convolution cancels is of the order of its terms, here at most a few
units, so 2^-17 is taken of 1 + the terms.
"""
import numpy as np
import pytest
import torch

from oracle import layer_step

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
ROUND = {BF: 2.0 ** -8, F: 2.0 ** -24}
WORK = 2.0 ** -17


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd as mod
    return mod


def make(seed, n, H, P, N, G, K, dtype, ddt, pool=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    pool = n + 3 if pool is None else pool
    C = H * P + 2 * G * N
    s = dict(xbc=r(n, C).to(dtype), ring=r(pool, K, C).to(dtype), w=r(C, K) / K, b=0.1 * r(C), dt=r(n, H).to(ddt), dt_bias=r(H) - 1,
             A_log=torch.rand(H, generator=g) * 2, D=r(H), states=r(pool, H, P, N), slots=torch.randperm(pool, generator=g)[:n].to(torch.int32),
             pos=torch.randint(0, 9, (n,), generator=g).to(torch.int32))
    return {k: v.cuda() for k, v in s.items()}


def call(ssd, s, G, **kw):
    return ssd.conv_scan_step(s["xbc"], s["ring"], s["w"], s["b"], s["dt"], s["dt_bias"], s["A_log"], s["D"], s["states"], s["slots"],
                              s["pos"], ngroups=G, **kw)


def oracle_of(s, G):
    return layer_step.conv_scan_step(s["xbc"], s["ring"], s["w"], s["b"], s["dt"], s["dt_bias"], s["A_log"], s["D"], s["states"], s["slots"],
                                     s["pos"], G)


def check(ssd, s, G, **kw):
    y0, ring, states, size = oracle_of(s, G)
    y = call(ssd, s, G, **kw)
    got = y.double().cpu().numpy()
    assert (np.abs(got - y0) <= ROUND[y.dtype] * np.abs(y0) + WORK * (size + (size > 0))).all(), np.abs(got - y0).max()
    st = s["states"].double().cpu().numpy()
    assert (np.abs(st - states) <= WORK * (1 + np.abs(states))).all(), np.abs(st - states).max()
    assert np.array_equal(s["ring"].double().cpu().numpy(), ring)
    return y


SHAPES = [  # rows, H, P, N, G, K
    (1, 1, 1, 4, 1, 2), (1, 80, 64, 128, 1, 4), (5, 24, 64, 128, 1, 4), (3, 8, 64, 128, 2, 4), (7, 6, 48, 20, 3, 3), (2, 5, 80, 256, 1, 4),
    (2, 4, 128, 512, 2, 2), (9, 7, 33, 64, 7, 4), (4, 2, 200, 16, 1, 3), (3, 4, 64, 132, 1, 4),
]


@pytest.mark.parametrize("dtype,ddt", [(BF, BF), (BF, F), (F, F)])
@pytest.mark.parametrize("n,H,P,N,G,K", SHAPES)
def test_shapes(ssd, n, H, P, N, G, K, dtype, ddt):
    check(ssd, make(1, n, H, P, N, G, K, dtype, ddt), G)


@pytest.mark.parametrize("dtype", [BF, F])
def test_views_of_one_projection(ssd, dtype):
    """xbc and dt as slices of the projection's rows, at odd offsets; y in a wider buffer whose rest stays."""
    n, H, P, N, G, K = 6, 5, 24, 36, 1, 4
    s = make(2, n, H, P, N, G, K, dtype, dtype)
    C = s["xbc"].shape[1]
    proj = torch.randn(n, 7 + C + H + 2, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    s["xbc"], s["dt"] = proj[:, 7:7 + C], proj[:, 7 + C:7 + C + H]
    buf = torch.full((n, H * P + 3), 5.0, dtype=dtype, device="cuda")
    check(ssd, s, G, y=buf[:, 1:1 + H * P].view(n, H, P))
    assert (buf[:, 0] == 5).all() and (buf[:, 1 + H * P:] == 5).all()


def test_padding_and_fresh_sequences(ssd):
    """Padding rows give zeros and touch nothing; a sequence at position 0 reads neither ring nor state (NaN there)."""
    n, H, P, N, G, K = 8, 4, 32, 64, 1, 4
    s = make(4, n, H, P, N, G, K, BF, BF)
    s["slots"][1], s["slots"][2], s["pos"][3], s["pos"][4] = -1, s["states"].shape[0], -5, 0
    s["slots"][5], s["pos"][5], s["pos"][6] = 2 ** 31 - 1, 2 ** 31 - 1, 2
    fresh = s["slots"][4].long()
    untouched = [i for i in range(s["states"].shape[0]) if i not in s["slots"][[0, 4, 6, 7]].tolist()]
    before = s["states"][untouched].clone(), s["ring"][untouched].clone()
    keep = s["states"][fresh].clone()
    s["states"][fresh] = float("nan")
    s["ring"][fresh] = float("nan")
    t = {k: v.clone() for k, v in s.items()}
    t["states"][fresh], t["ring"][fresh] = 0, 0
    y0, _, states, size = oracle_of(t, G)
    y = call(ssd, s, G)
    assert not y[[1, 2, 3, 5]].any()
    got = y.double().cpu().numpy()
    assert (np.abs(got - y0) <= ROUND[BF] * np.abs(y0) + WORK * (1 + size)).all()
    assert torch.equal(s["states"][untouched], before[0]) and torch.equal(s["ring"][untouched], before[1])
    assert np.allclose(s["states"][fresh].cpu().numpy(), states[fresh.item()], atol=1e-4) and keep.shape == s["states"][fresh].shape
    assert torch.equal(s["ring"][fresh, 0], s["xbc"][4]) and s["ring"][fresh, 1:].isnan().all()


@pytest.mark.parametrize("K", [2, 3, 4])
def test_position_near_the_end_of_its_range(ssd, K):
    s = make(5, 3, 2, 16, 16, 1, K, F, F)
    s["pos"][:] = torch.tensor([2 ** 31 - 1, 2 ** 31 - 2, K - 1])
    check(ssd, s, 1)


@pytest.mark.parametrize("dtype", [BF, F])
def test_prompt_then_tokens(ssd, dtype):
    """A prompt through the conv and scan calls, its states put into the pool, then tokens one at a time: as the whole
    sequence through the conv and scan calls in one go.  bf16: x, B and C are rounded between conv and scan there and not
    here, 2^-8 of the terms, which the sums over N and the recurrence average: 2^-6 of the largest y."""
    H, P, N, G, K, L, more = 4, 64, 128, 1, 4, 70, 6
    g = torch.Generator().manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    C = H * P + 2 * G * N
    xbc, dt = r(2, L + more, C).to(dtype), r(2, L + more, H)
    w, b, dt_bias, A_log, D = r(C, K) / K, r(C) * 0.1, r(H) - 1, r(H) * 0.3, r(H)

    def whole(n):
        x, B, Cm, cs = ssd.conv1d_silu_fwd(xbc[:, :n].contiguous(), w, b, nheads=H, headdim=P, ngroups=G, dstate=N)
        y, final = ssd.ssd_scan_fwd(x, dt[:, :n].contiguous(), dt_bias, A_log, B, Cm, D, chunk=64)
        return y, final, cs

    ref = whole(L + more)[0]
    _, final, cs = whole(L)
    ring, states = torch.full((5, K, C), float("nan"), dtype=dtype, device="cuda"), torch.full((5, H, P, N), float("nan"), device="cuda")
    slots = torch.tensor([3, 1], device="cuda")
    states[slots] = final
    ssd.conv_ring_store(ring, cs, slots, torch.full((2,), L, device="cuda"))
    for t in range(L, L + more):
        y = ssd.conv_scan_step(xbc[:, t], ring, w, b, dt[:, t], dt_bias, A_log, D, states, slots.int(),
                               torch.full((2,), t, dtype=torch.int32, device="cuda"), ngroups=G)
        tol = 2.0 ** -6 if dtype == BF else 2.0 ** -15
        assert (y.float() - ref[:, t].float()).abs().max() <= tol * ref.float().abs().max()


def test_states_past_32_bits(ssd):
    """Slots whose states lie past 2^32 bytes and 2^31 elements."""
    H, P, N, K = 32, 128, 512, 4
    pool = (1 << 31) // (H * P * N) + 3
    s = make(7, 2, H, P, N, 1, K, BF, BF, pool=3)
    big = torch.empty(pool, H, P, N, device="cuda")
    ring = torch.empty(pool, K, s["ring"].shape[2], dtype=BF, device="cuda")
    at = torch.tensor([pool - 1, pool - 2], device="cuda")
    big[at], ring[at] = s["states"][s["slots"].long()], s["ring"][s["slots"].long()]
    y = call(ssd, dict(s, states=big, ring=ring, slots=at.int()), 1)
    y2 = call(ssd, s, 1)
    assert torch.equal(y, y2) and torch.equal(big[at], s["states"][s["slots"].long()]) and torch.equal(ring[at], s["ring"][s["slots"].long()])


def test_no_rows(ssd):
    s = make(8, 0, 2, 8, 8, 1, 4, F, F)
    assert call(ssd, s, 1).shape == (0, 2, 8)
