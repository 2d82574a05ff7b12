"""GPU parity of the residual norm, the 8-bit norms and the norm's gradients.

Tolerances, per element, from the arithmetic: one rounding of the result (2^-8 |ref| for bf16, 2^-24 for fp32) and the
fp32 work behind it.  A sum of squares is at most 16 additions in a thread, then two trees of 5: below 2^-19 relative,
half of that in its root; with the products behind it 2^-18 of the terms' magnitude.  The gate's exponential is within
2 + 1.16 |z| units of 2^-23: 2^-16 of the term where |z| < 100.  8-bit values: within half a step, and 127 times the
relative error of v / scale (2^-15 with both of them).  The weight's gradient adds at most 36 rows in a block here and
up to 40 blocks' partials in a row, then a tree: 2^-17 of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

from oracle import layer_step

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
ROUND = {BF: 2.0 ** -8, F: 2.0 ** -24}
WORK, GATE, SUMS = 2.0 ** -18, 2.0 ** -16, 2.0 ** -17
EPS = 1e-5
DIMS = [8, 24, 256, 264, 520, 1000, 1024, 1032, 2560, 4096, 4104, 8192, 16384]


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd as mod
    return mod


def normal(seed, *shape, dtype=F):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def weight(seed, D):
    return 1.0 + 0.3 * normal(seed, D)


def near(got, ref, dtype, terms):
    got = got.double().cpu().numpy()
    assert (np.abs(got - ref) <= ROUND[dtype] * np.abs(ref) + terms + 1e-37).all(), np.abs(got - ref).max()


def check_q8(q, scale, v, rel):
    want = layer_step.q8_scale(v)
    s = scale.double().cpu().numpy()
    assert (np.abs(s - want) <= rel * want).all()
    steps = np.divide(v, want[:, None], out=np.zeros_like(v), where=want[:, None] > 0)
    assert (np.abs(q.cpu().numpy() - steps) <= 0.5 + 2 * 127 * rel).all()
    assert q.abs().max() <= 127


@pytest.mark.parametrize("dtype,rdtype", [(BF, None), (BF, BF), (BF, F), (F, None), (F, F)])
@pytest.mark.parametrize("D", DIMS)
def test_forward(ssd, D, dtype, rdtype):
    n = 1 if D == 16384 else 19
    x, w = normal(1, n, D, dtype=dtype), weight(2, D)
    res = None if rdtype is None else 3 * normal(3, n, D, dtype=rdtype)
    ref, h = layer_step.add_rmsnorm(x, w, res, EPS)
    size = np.abs(ref) if res is None else layer_step.inv_rms(h, EPS) * (np.abs(x.double().cpu().numpy()) + np.abs(res.double().cpu().numpy())) * np.abs(w.double().cpu().numpy())
    out, ro = ssd.add_rmsnorm_fwd(x, w, res, eps=EPS)
    near(out, ref, dtype, WORK * size)
    q, scale, ro8 = ssd.add_rmsnorm_q8_fwd(x, w, res, eps=EPS)
    check_q8(q, scale, ref, 2 * WORK)
    if res is None:
        assert ro is None and ro8 is None
    else:
        near(ro, h, rdtype, 2.0 ** -24 * np.abs(h))
        assert torch.equal(ro, ro8)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("D", DIMS)
def test_gated(ssd, D, dtype):
    n = 19
    y, z, w = normal(4, n, D, dtype=dtype), 4 * normal(5, n, D, dtype=dtype), weight(6, D)
    ref, _ = layer_step.add_rmsnorm(y, w, None, EPS, gate=z)
    q, scale = ssd.gated_rmsnorm_q8_fwd(y, z, w, EPS)
    check_q8(q, scale, ref, GATE)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("D", [64, 1000, 2560, 8192])
def test_gate_as_a_slice_of_the_projection(ssd, D, dtype):
    """z at an odd offset, its rows an odd stride apart."""
    n = 11
    y, w, proj = normal(45, n, D, dtype=dtype), weight(46, D), normal(47, n, D + 13, dtype=dtype)
    q, scale = ssd.gated_rmsnorm_q8_fwd(y, proj[:, 5:5 + D], w, EPS)
    rq, rscale = ssd.gated_rmsnorm_q8_fwd(y, proj[:, 5:5 + D].contiguous(), w, EPS)
    assert torch.equal(q, rq) and torch.equal(scale, rscale)


@pytest.mark.parametrize("dtype,rdtype,with_res", [(BF, BF, True), (BF, F, True), (BF, BF, False), (F, F, True), (F, F, False)])
@pytest.mark.parametrize("n,D", [(1, 8), (37, 264), (700, 1000), (5, 1032), (1500, 2560), (65, 4104), (3, 16384), (9000, 64)])
def test_gradients(ssd, n, D, dtype, rdtype, with_res):
    h, d, w = 2 * normal(7, n, D, dtype=rdtype), normal(8, n, D, dtype=dtype), weight(9, D)
    dr = normal(10, n, D, dtype=rdtype) if with_res else None
    dx, dw = ssd.add_rmsnorm_bwd(h, w, d, dr, eps=EPS)
    rx, rw, sx, sw = layer_step.add_rmsnorm_grad(h, w, d, dr, EPS)
    near(dx, rx, rdtype, WORK * sx)
    near(dw, rw, F, SUMS * sw)
    again = ssd.add_rmsnorm_bwd(h, w, d, dr, eps=EPS)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    ws = torch.empty(ssd.add_rmsnorm_bwd_workspace_size(h, d), dtype=torch.uint8, device="cuda")
    own = ssd.add_rmsnorm_bwd(h, w, d, dr, eps=EPS, workspace=ws)
    assert torch.equal(dx, own[0]) and torch.equal(dw, own[1])


def test_gradients_agree_with_differences_of_the_kernel(ssd):
    """fp32: the loss' change along a direction, by central differences of the forward (steps of 2^-7: the cubic term and
    the rounding are both below 2^-9 of it)."""
    n, D = 4, 64
    x, r, w, d, dr, u = (normal(20 + i, n, D) for i in range(6))
    w = weight(30, D)
    dx, _ = ssd.add_rmsnorm_bwd(x + r, w, d, dr, eps=EPS)
    t = 2.0 ** -7

    def loss(x):
        out, h = ssd.add_rmsnorm_fwd(x, w, r, eps=EPS)
        return (out.double() * d).sum() + (h.double() * dr).sum()

    slope = ((loss(x + t * u) - loss(x - t * u)) / (2 * t)).item()
    assert abs(slope - (dx.double() * u).sum().item()) <= 2.0 ** -8 * (dx.double() * u).abs().sum().item()


@pytest.mark.parametrize("D", [64, 1000, 2560])
def test_views_and_in_place(ssd, D):
    n = 21
    big = normal(40, n, 2 * D + 16, dtype=BF)
    x, res = big[:, :D], big[:, D + 16:]
    w = weight(41, D)
    out, ro = ssd.add_rmsnorm_fwd(x.contiguous(), w, res.contiguous(), eps=EPS)
    q, scale, _ = ssd.add_rmsnorm_q8_fwd(x.contiguous(), w, res.contiguous(), eps=EPS)
    got, gro = ssd.add_rmsnorm_fwd(x, w, res, eps=EPS)
    assert torch.equal(got, out) and torch.equal(gro, ro)
    qb = torch.full((n, D + 40), 99, dtype=torch.int8, device="cuda")
    sb = torch.full((n + 2,), 9.0, device="cuda")
    ssd.add_rmsnorm_q8_fwd(x, w, res, eps=EPS, q=qb[:, 8:8 + D], scale=sb[1:-1], return_residual=False)
    assert torch.equal(qb[:, 8:8 + D], q) and torch.equal(sb[1:-1], scale)
    assert (qb[:, :8] == 99).all() and (qb[:, 8 + D:] == 99).all() and sb[0] == 9 and sb[-1] == 9
    keep = big.clone()
    ssd.add_rmsnorm_fwd(x, w, res, eps=EPS, out=x, residual_out=res)   # both in place, in one buffer
    assert torch.equal(x, out) and torch.equal(res, ro) and torch.equal(big[:, D:D + 16], keep[:, D:D + 16])
    h, d, dr = normal(42, n, D, dtype=BF), normal(43, n, D, dtype=BF), normal(44, n, D, dtype=BF)
    dx, dw = ssd.add_rmsnorm_bwd(h, w, d, dr, eps=EPS)
    for name in ("d", "dr"):
        t = dict(d=d.clone(), dr=dr.clone())
        gx, gw = ssd.add_rmsnorm_bwd(h, w, t["d"], t["dr"], eps=EPS, dx=t[name])
        assert torch.equal(gx, dx) and torch.equal(gw, dw)


@pytest.mark.parametrize("D", [256, 2560])
@pytest.mark.parametrize("dtype", [BF, F])
def test_rows_that_hold_nothing_or_no_number(ssd, D, dtype):
    """Zeros stay zeros with eps 0, and have zero gradients; a row with an infinity or NaN gives scale NaN and q 0, and other rows do not see it."""
    x, w = normal(50, 6, D, dtype=dtype), weight(51, D)
    x[1] = 0
    x[2, 7], x[3, D - 1], x[4, 0] = float("inf"), float("nan"), -float("inf")
    out, _ = ssd.add_rmsnorm_fwd(x, w, eps=0.0)
    q, scale, _ = ssd.add_rmsnorm_q8_fwd(x, w, eps=0.0)
    assert not out[1].any() and not q[1].any() and scale[1] == 0
    assert not q[2:5].any() and scale[2:5].isnan().all() and out[2:5].isnan().any(1).all()
    ref, _ = layer_step.add_rmsnorm(x[[0, 5]], w, None, 0.0)
    near(out[[0, 5]], ref, dtype, WORK * np.abs(ref))
    check_q8(q[[0, 5]], scale[[0, 5]], ref, 2 * WORK)
    bad = weight(52, D)
    bad[3] = float("nan")
    q, scale, _ = ssd.add_rmsnorm_q8_fwd(x[[0, 5]].contiguous(), bad, eps=0.0)
    assert scale.isnan().all() and not q.any()
    q, scale = ssd.gated_rmsnorm_q8_fwd(x, torch.ones_like(x), w, 0.0)
    assert not q[1:5].any() and scale[1] == 0 and scale[2:5].isnan().all() and scale[[0, 5]].isfinite().all()
    h, d = normal(53, 2, D, dtype=dtype), normal(54, 2, D, dtype=dtype)
    h[1] = 0
    dx, dw = ssd.add_rmsnorm_bwd(h, w, d, eps=0.0)
    rx, rw, sx, sw = layer_step.add_rmsnorm_grad(h, w, d, None, 0.0)
    near(dx, rx, dtype, WORK * sx)
    near(dw, rw, F, SUMS * sw)


def test_tiny_and_large_values(ssd):
    D = 512
    x = normal(60, 4, D) * torch.tensor([1e-12, 1e12, 1.0, 1.0], device="cuda")[:, None]
    w = weight(61, D)
    q, scale, _ = ssd.add_rmsnorm_q8_fwd(x, w, eps=0.0)
    ref, _ = layer_step.add_rmsnorm(x, w, None, 0.0)
    check_q8(q, scale, ref, 2 * WORK)
    q, scale, _ = ssd.add_rmsnorm_q8_fwd(x, w * 1e-38, eps=0.0)   # scales below 2^-126: zero
    assert not q.any() and not scale.any()


def test_no_rows(ssd):
    x, w = torch.empty(0, 64, dtype=BF, device="cuda"), weight(70, 64)
    out, ro = ssd.add_rmsnorm_fwd(x, w, x.clone())
    q, scale, _ = ssd.add_rmsnorm_q8_fwd(x, w)
    dw = torch.ones(64, device="cuda")
    dx, _ = ssd.add_rmsnorm_bwd(x, w, x, dweight=dw)
    assert out.shape == ro.shape == q.shape == dx.shape == (0, 64) and scale.shape == (0,)
    assert not dw.any()


def test_rows_past_32_bits(ssd):
    """A row stride that puts the last rows past 2^32 elements."""
    D, stride = 64, (1 << 31) + 64
    big = torch.empty(2 * stride + D, dtype=BF, device="cuda")
    x = big.as_strided((3, D), (stride, 1))
    x.copy_(normal(80, 3, D, dtype=BF))
    w = weight(81, D)
    a, b = ssd.add_rmsnorm_fwd(x, w, eps=EPS)[0], ssd.add_rmsnorm_fwd(x.contiguous(), w, eps=EPS)[0]
    assert torch.equal(a, b)
