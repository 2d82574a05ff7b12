"""CPU checks of the entry points around the scan: every refusal happens before any CUDA call (the pointers here are made
up), and tensors, a stream or a workspace of another device are refused by the binding."""
import pytest
import torch

from test_attn_layer_device import Fake, FakeStream, ssd as no_library  # noqa: F401  (a fixture)

INVALID, NULL, MISALIGNED, UNSUPPORTED, ALIASING, SCRATCH, DTYPE = 1, 2, 3, 4, 7, 8, 9
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def ssd():
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd as mod
    return mod


def at(i):
    """Made-up arrays 1 GiB apart."""
    return (i + 1) << 30


def fill(cls, base, kw):
    base = dict(base, **kw)
    return cls(*(base.get(f, 0) for f, _ in cls._fields_))


NORM = dict(rows=10, dim=64, dtype=BF16, residual_dtype=BF16, eps=1e-6, x_stride=64, z_stride=64, residual_stride=64, out_stride=64,
            ro_stride=64, q_stride=64)
FWD = ("x", "residual", "weight", "out", "q", "q_scale", "residual_out")
GATED = ("y", "z", "weight", "q", "q_scale")
BWD = ("h", "weight", "dout", "dresidual", "dx", "dweight", "workspace")


def fwd(ssd, ptrs=None, q8=False, **kw):
    p = {n: at(i) for i, n in enumerate(FWD)}
    p.update(dict(out=None) if q8 else dict(q=None, q_scale=None))
    p.update(ptrs or {})
    return ssd.lib().ssd_add_rmsnorm_fwd(*(p[n] for n in FWD), fill(ssd.SsdNormDims, NORM, kw), None)


def gated(ssd, ptrs=None, **kw):
    p = {n: at(i) for i, n in enumerate(GATED)}
    p.update(ptrs or {})
    return ssd.lib().ssd_gated_rmsnorm_q8_fwd(*(p[n] for n in GATED), fill(ssd.SsdNormDims, NORM, kw), None)


def bwd(ssd, ptrs=None, size=1 << 28, **kw):
    p = {n: at(i) for i, n in enumerate(BWD)}
    p.update(ptrs or {})
    return ssd.lib().ssd_add_rmsnorm_bwd(*(p[n] for n in BWD), size, fill(ssd.SsdNormDims, NORM, kw), None)


NORM_DIMS = [
    (dict(rows=-1), INVALID), (dict(rows=2 ** 31), INVALID), (dict(dim=0), INVALID), (dict(flags=1), INVALID), (dict(reserved=1), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(dtype=2), DTYPE), (dict(residual_dtype=3), DTYPE),
    (dict(dtype=F32, residual_dtype=BF16), DTYPE), (dict(dim=60), UNSUPPORTED), (dict(dim=16392), UNSUPPORTED),
    (dict(x_stride=-64), INVALID), (dict(x_stride=68), MISALIGNED), (dict(x_stride=2 ** 60), INVALID),
]


@pytest.mark.parametrize("kw,status", NORM_DIMS)
def test_norm_dims(ssd, kw, status):
    assert fwd(ssd, **kw) == fwd(ssd, q8=True, **kw) == gated(ssd, **kw) == bwd(ssd, **kw) == status


@pytest.mark.parametrize("kw,q8,status", [
    (dict(residual_stride=68), False, MISALIGNED), (dict(out_stride=68), False, MISALIGNED), (dict(out_stride=56), False, INVALID),
    (dict(ro_stride=0), False, INVALID), (dict(q_stride=56), True, INVALID), (dict(q_stride=68), True, MISALIGNED)])
def test_norm_forward_strides(ssd, kw, q8, status):
    assert fwd(ssd, q8=q8, **kw) == status


@pytest.mark.parametrize("ptrs,q8,status", [
    (dict(x=None), False, NULL), (dict(weight=None), False, NULL), (dict(residual=None), False, NULL), (dict(out=None), False, NULL),
    (dict(q=None), True, NULL), (dict(q_scale=None), True, NULL), (dict(out=at(3)), True, INVALID),
    (dict(x=at(0) + 8), False, MISALIGNED), (dict(residual=at(1) + 8), False, MISALIGNED), (dict(weight=at(2) + 4), False, MISALIGNED),
    (dict(out=at(3) + 2), False, MISALIGNED), (dict(residual_out=at(6) + 8), False, MISALIGNED), (dict(q=at(4) + 4), True, MISALIGNED),
    (dict(q_scale=at(5) + 2), True, MISALIGNED),
    (dict(out=at(0) + 16), False, ALIASING), (dict(out=at(1)), False, ALIASING), (dict(out=at(2)), False, ALIASING),
    (dict(residual_out=at(0)), False, ALIASING), (dict(residual_out=at(1) + 128), False, ALIASING), (dict(residual_out=at(3)), False, ALIASING),
    (dict(q=at(0)), True, ALIASING), (dict(q=at(6) + 64), True, ALIASING), (dict(q_scale=at(4)), True, ALIASING),
    (dict(q_scale=at(2) + 32), True, ALIASING)])
def test_norm_forward_pointers(ssd, ptrs, q8, status):
    assert fwd(ssd, ptrs, q8=q8) == status


@pytest.mark.parametrize("ptrs,status", [
    *[({n: None}, NULL) for n in GATED], *[({n: at(i) + 2}, MISALIGNED) for i, n in enumerate(GATED) if n != "z"],
    (dict(z=at(1) + 1), MISALIGNED),
    (dict(q=at(0)), ALIASING), (dict(q=at(1) + 64), ALIASING), (dict(q_scale=at(2)), ALIASING), (dict(q_scale=at(3)), ALIASING)])
def test_gated_pointers(ssd, ptrs, status):
    assert gated(ssd, ptrs) == status


@pytest.mark.parametrize("ptrs,kw,status", [
    *[({n: None}, {}, NULL) for n in ("h", "weight", "dout", "dx")], *[({n: at(i) + 8}, {}, MISALIGNED) for i, n in enumerate(BWD)],
    (dict(dx=at(0)), {}, ALIASING), (dict(dx=at(1)), {}, ALIASING), (dict(dx=at(3) + 16), {}, ALIASING),
    (dict(dx=at(2)), dict(residual_dtype=F32), ALIASING), (dict(dweight=at(1)), {}, ALIASING), (dict(dweight=at(4) + 16), {}, ALIASING),
    (dict(workspace=at(5)), {}, ALIASING), (dict(workspace=at(2)), {}, ALIASING),
    ({}, dict(out_stride=56), INVALID), ({}, dict(ro_stride=68), MISALIGNED), ({}, dict(residual_stride=-8), INVALID), ({}, dict(size=255), SCRATCH)])
def test_norm_backward(ssd, ptrs, kw, status):
    assert bwd(ssd, ptrs, **kw) == status


def test_null_dims_and_sizes(ssd):
    lib = ssd.lib()
    assert lib.ssd_add_rmsnorm_fwd(*[at(i) for i in range(7)], None, None) == NULL
    assert lib.ssd_gated_rmsnorm_q8_fwd(*[at(i) for i in range(5)], None, None) == NULL
    assert lib.ssd_add_rmsnorm_bwd(*[at(i) for i in range(7)], 0, None, None) == NULL
    assert lib.ssd_q8_matmul(*[at(i) for i in range(6)], 0, None, None) == NULL
    assert lib.ssd_q8_pack_weight(at(0), at(1), None, None) == NULL
    assert lib.ssd_conv_scan_step(*[at(i) for i in range(12)], None, None) == NULL
    assert lib.ssd_add_rmsnorm_bwd_workspace_size(fill(ssd.SsdNormDims, NORM, {}), None) == NULL
    assert lib.ssd_q8_matmul_workspace_size(fill(ssd.SsdQ8Dims, Q8, {}), None) == NULL


Q8 = dict(M=10, N=100, K=70, out_dtype=BF16, a_stride=70, y_stride=100)
Q8_ARGS = ("a", "a_scale", "packed", "w_scale", "y", "workspace")


def q8(ssd, ptrs=None, size=1 << 28, **kw):
    p = {n: at(i) for i, n in enumerate(Q8_ARGS)}
    p.update(ptrs or {})
    return ssd.lib().ssd_q8_matmul(*(p[n] for n in Q8_ARGS), size, fill(ssd.SsdQ8Dims, Q8, kw), None)


@pytest.mark.parametrize("kw,ptrs,status", [
    (dict(M=-1), {}, INVALID), (dict(M=2 ** 31), {}, INVALID), (dict(N=0), {}, INVALID), (dict(N=2 ** 24 + 1), {}, INVALID),
    (dict(K=0), {}, INVALID), (dict(K=65537, a_stride=65537), {}, UNSUPPORTED), (dict(flags=1), {}, INVALID), (dict(out_dtype=2), {}, DTYPE),
    (dict(a_stride=-1), {}, INVALID), (dict(y_stride=99), {}, INVALID), (dict(y_stride=2 ** 60), {}, INVALID),
    *[({}, {n: None}, NULL) for n in Q8_ARGS[:5]],
    ({}, dict(a_scale=at(1) + 2), MISALIGNED), ({}, dict(packed=at(2) + 8), MISALIGNED), ({}, dict(w_scale=at(3) + 1), MISALIGNED),
    ({}, dict(y=at(4) + 1), MISALIGNED), (dict(out_dtype=F32), dict(y=at(4) + 2), MISALIGNED), ({}, dict(workspace=at(5) + 8), MISALIGNED),
    ({}, dict(y=at(0) + 690), ALIASING), ({}, dict(y=at(1)), ALIASING), ({}, dict(y=at(2) + 64), ALIASING), ({}, dict(y=at(3)), ALIASING),
    ({}, dict(workspace=at(4)), ALIASING), ({}, dict(workspace=at(2)), ALIASING)])
def test_q8_matmul(ssd, kw, ptrs, status):
    assert q8(ssd, ptrs, **kw) == status


@pytest.mark.parametrize("kw,ptrs,status", [
    (dict(N=0), {}, INVALID), (dict(K=0), {}, INVALID), (dict(a_stride=69), {}, INVALID), ({}, dict(w=None), NULL), ({}, dict(packed=None), NULL),
    ({}, dict(packed=at(1) + 8), MISALIGNED), ({}, dict(w=at(1) + 100), ALIASING)])
def test_q8_pack(ssd, kw, ptrs, status):
    p = dict(dict(w=at(0), packed=at(1)), **ptrs)
    assert ssd.lib().ssd_q8_pack_weight(p["w"], p["packed"], fill(ssd.SsdQ8Dims, Q8, kw), None) == status


STEP = dict(rows=5, nslots=7, nheads=4, headdim=16, dstate=8, ngroups=2, kernel_size=4, dtype=BF16, dt_dtype=F32, xbc_stride=96, dt_stride=4,
            y_stride=64)
STEP_ARGS = ("xbc", "ring", "weight", "bias", "dt_raw", "dt_bias", "A_log", "D", "states", "slots", "positions", "y")


def step(ssd, ptrs=None, **kw):
    p = {n: at(i) for i, n in enumerate(STEP_ARGS)}
    p.update(ptrs or {})
    return ssd.lib().ssd_conv_scan_step(*(p[n] for n in STEP_ARGS), fill(ssd.SsdStepDims, STEP, kw), None)


@pytest.mark.parametrize("kw,ptrs,status", [
    (dict(rows=-1), {}, INVALID), (dict(nslots=-1), {}, INVALID), (dict(nslots=2 ** 31), {}, INVALID), (dict(nheads=0), {}, INVALID),
    (dict(nheads=5), {}, INVALID), (dict(headdim=0), {}, INVALID), (dict(ngroups=0), {}, INVALID), (dict(flags=1), {}, INVALID),
    (dict(dstate=10), {}, UNSUPPORTED), (dict(dstate=516), {}, UNSUPPORTED), (dict(kernel_size=1), {}, UNSUPPORTED),
    (dict(kernel_size=5), {}, UNSUPPORTED), (dict(headdim=2049), {}, UNSUPPORTED), (dict(rows=2 ** 29), {}, UNSUPPORTED),
    (dict(dtype=2), {}, DTYPE), (dict(dt_dtype=2), {}, DTYPE), (dict(dtype=F32, dt_dtype=BF16), {}, DTYPE),
    (dict(xbc_stride=-1), {}, INVALID), (dict(y_stride=63), {}, INVALID), (dict(dt_stride=2 ** 61), {}, INVALID),
    *[({}, {n: None}, NULL) for n in STEP_ARGS if n != "bias"],
    *[({}, {n: at(i) + 1}, MISALIGNED) for i, n in enumerate(STEP_ARGS)],
    *[({}, {n: at(i) + 8}, MISALIGNED) for i, n in enumerate(STEP_ARGS) if n in ("ring", "weight", "states")],
    ({}, dict(y=at(0)), ALIASING), ({}, dict(y=at(8) + 64), ALIASING), ({}, dict(y=at(1)), ALIASING), ({}, dict(ring=at(0)), ALIASING),
    ({}, dict(ring=at(8) + 4096), ALIASING), ({}, dict(states=at(2)), ALIASING), ({}, dict(slots=at(8) + 4), ALIASING),
    ({}, dict(positions=at(11) + 4), ALIASING)])
def test_step(ssd, kw, ptrs, status):
    assert step(ssd, ptrs, **kw) == status


def calls(ssd, dev, **kw):
    t = lambda *s, dtype=torch.bfloat16: Fake(*s, dtype=dtype, device=dev)  # noqa: E731
    f = lambda *s: t(*s, dtype=torch.float32)  # noqa: E731
    i, b = (lambda *s: t(*s, dtype=torch.int32)), (lambda *s: t(*s, dtype=torch.int8))  # noqa: E731
    yield lambda: ssd.add_rmsnorm_fwd(t(4, 64), f(64), t(4, 64), out=t(4, 64), residual_out=t(4, 64), **kw)
    yield lambda: ssd.add_rmsnorm_q8_fwd(t(4, 64), f(64), t(4, 64), q=b(4, 64), scale=f(4), residual_out=t(4, 64), **kw)
    yield lambda: ssd.gated_rmsnorm_q8_fwd(t(4, 64), t(4, 64), f(64), q=b(4, 64), scale=f(4), **kw)
    yield lambda: ssd.add_rmsnorm_bwd(t(4, 64), f(64), t(4, 64), t(4, 64), dx=t(4, 64), dweight=f(64), **kw)
    yield lambda: ssd.q8_pack_weight(b(128, 64), packed=b(8192), **kw)
    yield lambda: ssd.q8_matmul(b(4, 64), f(4), b(8192), f(128), out=t(4, 128), **kw)
    yield lambda: ssd.conv_scan_step(t(4, 64), t(6, 4, 64), f(64, 4), f(64), f(4, 2), f(2), f(2), f(2), f(6, 2, 16, 16), i(4), i(4),
                                     ngroups=1, y=t(4, 2, 16), **kw)


@pytest.mark.parametrize("k", range(7))
def test_another_device(no_library, k):  # noqa: F811
    for _ in range(2):   # (a remembered layout too)
        with pytest.raises(ValueError, match="not the current device"):
            list(calls(no_library, "cuda:1"))[k]()
    with pytest.raises(ValueError, match="the stream is not"):
        list(calls(no_library, "cuda:0", stream=FakeStream(1)))[k]()
    with pytest.raises(AssertionError, match="was reached"):
        list(calls(no_library, "cuda:0", stream=FakeStream(0)))[k]()


def bad_calls(ssd):
    t = lambda *s, dtype=torch.bfloat16: Fake(*s, dtype=dtype, device="cuda:0")  # noqa: E731
    f = lambda *s: t(*s, dtype=torch.float32)  # noqa: E731
    i, b = (lambda *s: t(*s, dtype=torch.int32)), (lambda *s: t(*s, dtype=torch.int8))  # noqa: E731
    x, w = t(4, 64), f(64)
    yield lambda: ssd.add_rmsnorm_fwd(t(4, 2, 64), w)
    yield lambda: ssd.add_rmsnorm_fwd(x, f(32))
    yield lambda: ssd.add_rmsnorm_fwd(x, t(64))
    yield lambda: ssd.add_rmsnorm_fwd(x, w, t(5, 64))
    yield lambda: ssd.add_rmsnorm_fwd(x, w, out=f(4, 64))
    yield lambda: ssd.add_rmsnorm_fwd(x, w, residual_out=t(4, 64))
    yield lambda: ssd.add_rmsnorm_q8_fwd(x, w, q=t(4, 64))
    yield lambda: ssd.add_rmsnorm_q8_fwd(x, w, scale=f(5))
    yield lambda: ssd.gated_rmsnorm_q8_fwd(x, t(4, 32), w)
    yield lambda: ssd.gated_rmsnorm_q8_fwd(x, f(4, 64), w)
    yield lambda: ssd.add_rmsnorm_bwd(x, w, t(4, 32))
    yield lambda: ssd.add_rmsnorm_bwd(x, w, x, f(4, 64))
    yield lambda: ssd.add_rmsnorm_bwd(x, w, x, dweight=f(32))
    yield lambda: ssd.q8_pack_weight(t(128, 64))
    yield lambda: ssd.q8_pack_weight(b(128, 64), packed=b(100))
    yield lambda: ssd.q8_matmul(t(4, 64), f(4), b(8192), f(128))
    yield lambda: ssd.q8_matmul(b(4, 64), f(5), b(8192), f(128))
    yield lambda: ssd.q8_matmul(b(4, 64), f(4), b(8191), f(128))
    yield lambda: ssd.q8_matmul(b(4, 64), f(4), b(8192), f(128), out=t(4, 127))
    step = dict(xbc=t(4, 64), conv_ring=t(6, 4, 64), weight=f(64, 4), bias=None, dt_raw=f(4, 2), dt_bias=f(2), A_log=f(2), D=f(2),
                states=f(6, 2, 16, 16), slots=i(4), positions=i(4), ngroups=1)
    for name, bad in (("xbc", t(4, 60)), ("conv_ring", f(6, 4, 64)), ("conv_ring", t(5, 4, 64)), ("weight", f(60, 4)), ("bias", f(60)),
                      ("dt_raw", f(4, 3)), ("D", f(3)), ("states", t(6, 2, 16, 16)), ("slots", i(5)), ("positions", t(4, dtype=torch.int64)),
                      ("ngroups", 2), ("y", f(4, 2, 16))):
        yield lambda name=name, bad=bad: ssd.conv_scan_step(**{**step, name: bad})


@pytest.mark.parametrize("k", range(31))
def test_wrong_tensors(no_library, k):  # noqa: F811
    with pytest.raises(ValueError):
        list(bad_calls(no_library))[k]()


def test_wrong_types(no_library):  # noqa: F811
    half = Fake(4, 64, dtype=torch.float16, device="cuda:0")
    w = Fake(64, dtype=torch.float32, device="cuda:0")
    with pytest.raises(no_library.SsdError):
        no_library.add_rmsnorm_fwd(half, w)
    with pytest.raises(no_library.SsdError):
        no_library.q8_matmul(Fake(4, 64, dtype=torch.int8, device="cuda:0"), w, w, w, dtype=torch.float16)
