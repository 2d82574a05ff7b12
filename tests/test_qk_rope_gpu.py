"""GPU parity of the q/k norm with rotary position and of its gradients.

Tolerances, per element, from the arithmetic: one rounding of the result (2^-8
|ref| for bf16, 2^-22 |ref| for fp32, twice the half-ulp) plus 2^-19 of the
magnitude of the terms behind it (a dozen fp32 operations on them, the sum of
256 squares among them).  A weight gradient is a sum in fp32 of at most a few
hundred sequential additions, then trees: 2^-15 of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

from oracle.attention import qk_norm_rope, qk_norm_rope_grad

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
ROUND = {BF: 2.0 ** -8, F: 2.0 ** -22}
TERMS, SUMS = 2.0 ** -19, 2.0 ** -15

SHAPES = [  # T, Hq, Hk, D, R, interleaved
    (1, 1, 1, 64, 64, False),
    (5, 32, 8, 128, 128, False),
    (37, 32, 8, 128, 128, True),
    (130, 20, 4, 80, 32, True),
    (33, 6, 2, 80, 80, False),
    (9, 3, 3, 96, 48, False),
    (17, 8, 1, 256, 256, False),
    (17, 8, 1, 192, 64, True),
    (11, 2, 2, 64, 0, False),
    (700, 5, 1, 64, 32, False),
    (3, 7, 2, 8, 0, True),
    (3, 7, 2, 24, 16, False),
    (6, 3, 2, 200, 16, False),
]


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd as mod
    return mod


def make(seed, T, Hq, Hk, D, R, dtype, max_pos=512):
    rng = np.random.default_rng(seed)
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    qkv = (f(T, Hq + 2 * Hk, D) * torch.from_numpy(rng.uniform(0.1, 4, (1, Hq + 2 * Hk, 1)).astype(np.float32))).to(dtype)
    pos = rng.integers(0, max_pos, T)
    pos[rng.random(T) < 0.1] = -1
    if T > 20:
        pos[7], pos[11] = max_pos, 2 ** 31 - 1   # outside the table: padding too
    freq = 10000.0 ** (-2.0 * np.arange(R // 2) / max(R, 1))
    ang = np.arange(max_pos)[:, None] * freq[None, :]
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a.astype(np.float32)))  # noqa: E731
    return dict(qkv=qkv, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hk], v=qkv[:, Hq + Hk:], qw=1 + 0.3 * f(D), kw=1 + 0.3 * f(D),
                cos=t(np.cos(ang)), sin=t(np.sin(ang)), pos=torch.from_numpy(pos.astype(np.int32)),
                dq=f(T, Hq, D).to(dtype), dk=f(T, Hk, D).to(dtype))


def on_gpu(c, Hq, Hk):
    qkv = c["qkv"].cuda()
    g = {k: v.cuda() for k, v in c.items() if k not in ("qkv", "q", "k", "v")}
    return dict(g, qkv=qkv, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hk], v=qkv[:, Hq + Hk:])


def near(got, ref, size, dtype):
    got = got.double().cpu().numpy()
    over = np.abs(got - ref) - (ROUND[dtype] * np.abs(ref) + TERMS * size)
    assert over.max(initial=-1) <= 0, f"off by {over.max()} over its bound"


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,Hq,Hk,D,R,inter", SHAPES)
def test_forward(ssd, dtype, T, Hq, Hk, D, R, inter):
    c = make(T + D, T, Hq, Hk, D, R, dtype)
    g = on_gpu(c, Hq, Hk)
    qo, ko = ssd.qk_norm_rope_fwd(g["q"], g["k"], g["qw"], g["kw"], g["cos"], g["sin"], g["pos"], eps=1e-5, interleaved=inter)
    torch.cuda.synchronize()
    for got, x, w in ((qo, c["q"], c["qw"]), (ko, c["k"], c["kw"])):
        ref, size = qk_norm_rope(x, w, c["cos"], c["sin"], c["pos"], 1e-5, inter)
        near(got, ref, size, dtype)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,Hq,Hk,D,R,inter", SHAPES)
def test_backward(ssd, dtype, T, Hq, Hk, D, R, inter):
    c = make(T + D + 1, T, Hq, Hk, D, R, dtype)
    g = on_gpu(c, Hq, Hk)
    got = ssd.qk_norm_rope_bwd(g["q"], g["k"], g["qw"], g["kw"], g["cos"], g["sin"], g["pos"], g["dq"], g["dk"], eps=1e-5,
                               interleaved=inter)
    torch.cuda.synchronize()
    for n, x, w in (("q", c["q"], c["qw"]), ("k", c["k"], c["kw"])):
        dx, dw, size, wsize = qk_norm_rope_grad(x, w, c["cos"], c["sin"], c["pos"], c["d" + n], 1e-5, inter)
        near(got["d" + n], dx, size, dtype)
        assert (np.abs(got[f"d{n}_weight"].double().cpu().numpy() - dw) <= SUMS * wsize).all()


@pytest.mark.parametrize("inter", [False, True])
def test_gradient_against_differences(ssd, inter):
    # fp32 gradients against central differences of the fp64 forward: step 1e-5, so the differences are
    # good to 1e-8; the gradients' own error is below 2^-19 of terms of a few units
    T, H, D, R = 3, 2, 32, 16
    c = make(77, T, H, H, D, R, F)
    c["pos"] = torch.tensor([5, -1, 300], dtype=torch.int32)
    g = on_gpu(c, H, H)
    got = ssd.qk_norm_rope_bwd(g["q"], g["k"], g["qw"], g["kw"], g["cos"], g["sin"], g["pos"], g["dq"], g["dk"], eps=1e-3,
                               interleaved=inter)
    torch.cuda.synchronize()
    x, w, dy = c["q"].double().numpy(), c["qw"].double().numpy(), c["dq"].double().numpy()

    def loss(x, w):
        return (qk_norm_rope(x, w, c["cos"], c["sin"], c["pos"], 1e-3, inter)[0] * dy).sum()

    h = 1e-5
    for at in [(0, 0, 0), (0, 1, 9), (0, 1, 31), (1, 0, 3), (2, 1, 15), (2, 0, 16)]:
        e = np.zeros_like(x)
        e[at] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - float(got["dq"][at])) < 2e-5
    for i in (0, 7, 8, 20, 31):
        e = np.zeros(D)
        e[i] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - float(got["dq_weight"][i])) < 2e-5


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "kv"])
@pytest.mark.parametrize("return_k", [False, True])
def test_into_the_cache(ssd, dtype, layout, return_k):
    T, Hq, Hk, D, R, ps, npages = 45, 6, 2, 80, 80, 7, 12
    c = make(5, T, Hq, Hk, D, R, dtype)
    g = on_gpu(c, Hq, Hk)
    shape = {"nhd": (npages, ps, Hk, D), "hnd": (npages, Hk, ps, D), "kv": (npages, 2, ps, Hk, D)}[layout]
    kc, vc = torch.full(shape, 3.0, dtype=dtype, device="cuda"), torch.full(shape, 3.0, dtype=dtype, device="cuda")
    if layout == "kv":
        kc, vc = kc[:, 0], kc[:, 1]
    elif layout == "hnd":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    rng = np.random.default_rng(1)
    slots = rng.permutation(npages * ps)[:T]
    slots[3], slots[8], slots[20] = -1, npages * ps, 2 ** 40   # not written
    qo, ko = ssd.qk_norm_rope_fwd(g["q"], g["k"], g["qw"], g["kw"], g["cos"], g["sin"], g["pos"], v=g["v"], k_cache=kc,
                                  v_cache=vc, slots=torch.from_numpy(slots).cuda(), return_k=return_k)
    torch.cuda.synchronize()
    ref, size = qk_norm_rope(c["k"], c["kw"], c["cos"], c["sin"], c["pos"], 1e-6, False)
    rq, qsize = qk_norm_rope(c["q"], c["qw"], c["cos"], c["sin"], c["pos"], 1e-6, False)
    near(qo, rq, qsize, dtype)
    assert (ko is not None) == return_k
    if return_k:
        near(ko, ref, size, dtype)
    live = (c["pos"].numpy() >= 0) & (c["pos"].numpy() < 512) & (slots >= 0) & (slots < npages * ps)
    kk, vv = np.full((npages * ps, Hk, D), 3.0), np.full((npages * ps, Hk, D), 3.0)
    ks = np.zeros((npages * ps, Hk, 1))
    kk[slots[live]], vv[slots[live]], ks[slots[live]] = ref[live], c["v"].double().numpy()[live], size[live]
    near(kc.reshape(npages * ps, Hk, D), kk, ks, dtype)
    assert np.array_equal(vc.reshape(npages * ps, Hk, D).double().cpu().numpy(), vv)


def test_in_place_and_strided_gradients(ssd):
    T, Hq, Hk, D = 40, 8, 2, 128
    c = make(6, T, Hq, Hk, D, D, BF)
    g = on_gpu(c, Hq, Hk)
    tab = (g["qw"], g["kw"], g["cos"], g["sin"], g["pos"])
    qo, ko = ssd.qk_norm_rope_fwd(g["q"], g["k"], *tab)
    ref = ssd.qk_norm_rope_bwd(g["q"], g["k"], *tab, g["dq"], g["dk"])
    # gradients into the views of a fused gradient, and over the incoming ones
    fused = torch.full((T, Hq + 2 * Hk, D), 9.0, dtype=BF, device="cuda")
    got = ssd.qk_norm_rope_bwd(g["q"], g["k"], *tab, g["dq"], g["dk"], dq=fused[:, :Hq], dk=fused[:, Hq:Hq + Hk])
    assert torch.equal(fused[:, :Hq], ref["dq"]) and torch.equal(fused[:, Hq:Hq + Hk], ref["dk"])
    assert (fused[:, Hq + Hk:] == 9).all() and torch.equal(got["dq_weight"], ref["dq_weight"])
    ws = torch.full((ssd.qk_norm_rope_bwd_workspace_size(g["q"], g["k"]),), 255, dtype=torch.uint8, device="cuda")
    got = ssd.qk_norm_rope_bwd(g["q"], g["k"], *tab, g["dq"], g["dk"], dq=g["dq"], dk=g["dk"], workspace=ws)
    for n in ref:
        assert torch.equal(got[n], ref[n])
    v = g["v"].clone()
    ssd.qk_norm_rope_fwd(g["q"], g["k"], *tab, q_out=g["q"], k_out=g["k"])
    assert torch.equal(g["q"], qo) and torch.equal(g["k"], ko) and torch.equal(g["v"], v)


def test_gradient_of_a_broadcast(ssd):
    # one incoming gradient shared by all heads (head stride 0)
    T, H, D = 30, 4, 64
    c = make(8, T, H, H, D, D, BF)
    g = on_gpu(c, H, H)
    d = g["dq"][:, :1]
    got = ssd.qk_norm_rope_bwd(g["q"], g["k"], g["qw"], None, g["cos"], g["sin"], g["pos"], d.expand(T, H, D), d.expand(T, H, D))
    ref = ssd.qk_norm_rope_bwd(g["q"], g["k"], g["qw"], None, g["cos"], g["sin"], g["pos"], d.repeat(1, H, 1), d.repeat(1, H, 1))
    torch.cuda.synchronize()
    for n in ref:
        assert torch.equal(got[n], ref[n])
    dk, dw, size, wsize = qk_norm_rope_grad(c["k"], None, c["cos"], c["sin"], c["pos"], c["dq"][:, :1].expand(T, H, D), 1e-6, False)
    near(got["dk"], dk, size, BF)
    assert (np.abs(got["dk_weight"].double().cpu().numpy() - dw) <= SUMS * wsize).all()


def test_no_tokens(ssd):
    c = make(9, 4, 4, 2, 64, 64, BF)
    g = on_gpu(c, 4, 2)
    z = lambda t: t[:0]  # noqa: E731
    tab = (g["qw"], g["kw"], g["cos"], g["sin"], z(g["pos"]))
    qo, ko = ssd.qk_norm_rope_fwd(z(g["q"]), z(g["k"]), *tab)
    assert qo.shape == (0, 4, 64) and ko.shape == (0, 2, 64)
    got = ssd.qk_norm_rope_bwd(z(g["q"]), z(g["k"]), *tab, z(g["dq"]), z(g["dk"]))
    torch.cuda.synchronize()
    assert (got["dq_weight"] == 0).all() and (got["dk_weight"] == 0).all()


def test_all_padding_and_nan_in_padding(ssd):
    T = 12
    c = make(10, T, 4, 2, 64, 64, BF)
    g = on_gpu(c, 4, 2)
    g["qkv"][:] = float("nan")
    g["dq"][:] = float("inf")
    pos = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    tab = (g["qw"], g["kw"], g["cos"], g["sin"], pos)
    kc = torch.full((2, 8, 2, 64), 5.0, dtype=BF, device="cuda")
    vc = kc.clone()
    qo, ko = ssd.qk_norm_rope_fwd(g["q"], g["k"], *tab, v=g["v"], k_cache=kc, v_cache=vc,
                                  slots=torch.arange(T, device="cuda"))
    got = ssd.qk_norm_rope_bwd(g["q"], g["k"], *tab, g["dq"], g["dk"])
    torch.cuda.synchronize()
    assert (qo == 0).all() and (ko == 0).all() and (kc == 5).all() and (vc == 5).all()
    assert all((got[n] == 0).all() for n in got)


def test_repeat_bits_and_rope_table(ssd):
    T, Hq, Hk, D = 3000, 8, 2, 128
    c = make(12, T, Hq, Hk, D, D, BF)
    g = on_gpu(c, Hq, Hk)
    cos, sin = ssd.rope_table(512, D)
    assert torch.equal(cos.cpu(), c["cos"]) and torch.equal(sin.cpu(), c["sin"])
    args = (g["q"], g["k"], g["qw"], g["kw"], cos, sin, g["pos"], g["dq"], g["dk"])
    a = ssd.qk_norm_rope_bwd(*args)
    for _ in range(3):
        b = ssd.qk_norm_rope_bwd(*args)
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_refusals(ssd):
    c = make(13, 16, 4, 2, 64, 64, BF)
    g = on_gpu(c, 4, 2)
    ok = dict(q=g["q"], k=g["k"], q_weight=g["qw"], k_weight=g["kw"], cos=g["cos"], sin=g["sin"], positions=g["pos"])
    kc = torch.zeros(4, 8, 2, 64, dtype=BF, device="cuda")
    slots = torch.arange(16, device="cuda")
    for bad in (dict(q=g["q"].half(), k=g["k"].half()), dict(k=g["k"].float()), dict(q=g["q"].cpu()), dict(positions=g["pos"].long()),
                dict(positions=g["pos"][:3]), dict(q_weight=g["qw"].bfloat16()), dict(k_weight=g["kw"][:32]),
                dict(cos=g["cos"][:, :30].contiguous(), sin=g["sin"][:, :30].contiguous()),     # rotary_dim 60
                dict(cos=torch.zeros(8, 40, device="cuda"), sin=torch.zeros(8, 40, device="cuda")),   # more than D
                dict(sin=g["sin"][:4]), dict(eps=-1.0), dict(q=g["q"][..., :60], k=g["k"][..., :60]),
                dict(return_k=False), dict(v=g["v"], k_cache=kc, v_cache=kc.clone()),
                dict(v=g["v"], k_cache=kc, v_cache=kc.clone(), slots=slots.int()),
                dict(v=g["v"], k_cache=kc[:, :, :1], v_cache=kc.clone(), slots=slots),
                dict(q_out=g["k"]), dict(q_out=g["qkv"][:, 1:5]), dict(k_out=g["v"], v=g["v"], k_cache=kc, v_cache=kc.clone(), slots=slots),
                dict(q_out=torch.zeros(16, 1, 64, dtype=BF, device="cuda").expand(16, 4, 64))):
        with pytest.raises((ValueError, ssd.SsdError)):
            ssd.qk_norm_rope_fwd(**dict(ok, **bad))
    with pytest.raises((ValueError, ssd.SsdError)):
        ssd.qk_norm_rope_bwd(*ok.values(), g["dq"], g["dk"], dq=g["q"])
    with pytest.raises((ValueError, ssd.SsdError)):
        ssd.qk_norm_rope_bwd(*ok.values(), g["dq"], g["dk"][:, :1])
