"""Which views of one buffer the attention layer's operators take: disjoint rows are
accepted however they interleave, shared bytes are refused.  The CPU cases (made-up
pointers) end in a refusal before any CUDA call; a workspace that is too small, which
is found after the checks of the views, stands for acceptance."""
import ctypes

import pytest
import torch

from test_attn_layer_abi import ALIASING, at, bwd, qk, qk_dims, ssd  # noqa: F401

SCRATCH = 8
W = 64 * 2   # bytes of a row: heads of 64, bf16


@pytest.mark.parametrize("kc,vc,off", [
    ((1024, 128, 64), (1024, 128, 64), 0),                 # one buffer as both caches
    ((1024, 128, 64), (1024, 128, 64), 7 * 1024 * 2),      # the last page of one is the first of the other
    ((2048, 128, 64), (2048, 128, 64), 512 * 2),           # halves of a page that reach into one another
    ((2048, 256, 64), (2048, 256, 64), 64 * 2),            # [page, token, 2 x 2 heads]: a head too far to the left
    ((1024, 64, 512), (1024, 128, 64), 1024),              # head-major over token-major
])
def test_caches_that_share_bytes_are_refused(ssd, kc, vc, off):
    assert qk(ssd, dict(k_cache=at(10), v_cache=at(10) + off), npages=8, kc_stride=kc, vc_stride=vc) == ALIASING


@pytest.mark.parametrize("name", ["kc_stride", "vc_stride"])
@pytest.mark.parametrize("strides", [(0, 128, 64), (1024, 0, 64), (1024, 128, 0), (512, 128, 64), (1024, 64, 64), (1024, 128, 32),
                                     (64, 64, 64)])
def test_cache_rows_that_share_bytes_are_refused(ssd, name, strides):
    assert qk(ssd, npages=8, **{name: strides}) == ALIASING


LAYOUTS = ["pkthd", "ptkhd", "pthkd", "pkhtd", "phtkd", "kpthd", "lpkthd", "plkthd", "tpkhd"]


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_caches_of_one_buffer(layout, dtype):
    # pages p, tokens t, heads h, keys and values k, layers l in any order (elements d innermost)
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd
    size = dict(p=6, t=8, h=2, k=2, l=3, d=64)
    buf = torch.full([size[x] for x in layout], 5.0, dtype=dtype, device="cuda")
    view = buf.permute([layout.index(x) for x in (["l"] if "l" in layout else []) + list("kpthd")])
    kc, vc = (view[1] if "l" in layout else view)
    T, Hq, Hk, D = 20, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = torch.randn(T, Hq + 2 * Hk, D, device="cuda", generator=g).to(dtype).split((Hq, Hk, Hk), 1)
    cos, sin = ssd.rope_table(64, D)
    slots = torch.randperm(48, device="cuda", generator=g)[:T]
    _, ko = ssd.qk_norm_rope_fwd(q, k, None, None, cos, sin, torch.arange(T, dtype=torch.int32, device="cuda"), v=v, k_cache=kc,
                                 v_cache=vc, slots=slots)
    torch.cuda.synchronize()
    want = torch.full((2, 6, 8, Hk, D), 5.0, dtype=dtype, device="cuda")
    want[0, slots // 8, slots % 8], want[1, slots // 8, slots % 8] = ko, v
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    assert int((buf != 5).sum()) == int((want != 5).sum())


def scratch(ssd, ptrs, **kw):
    """The backward with a workspace that is one byte short: found after the checks of the views, before any CUDA call."""
    n = ctypes.c_uint64(0)
    assert ssd.lib().ssd_qk_norm_rope_bwd_workspace_size(qk_dims(ssd, **kw), ctypes.byref(n)) == 0 and n.value > 0
    return bwd(ssd, ptrs, ws=(at(20), n.value - 1), **kw)


@pytest.mark.parametrize("ptrs,kw,status", [
    # gradients into a fused [token, head, q/k/v, 64] gradient: rows of one between rows of the other
    (dict(dq=at(9), dk=at(9) + W), dict(nheads_q=2, dq_stride=(384, 192), dk_stride=(384, 192)), SCRATCH),
    # ... and over the incoming gradients, views of another such buffer
    (dict(dq_out=at(9), dk_out=at(9) + W, dq=at(9), dk=at(9) + W),
     dict(nheads_q=2, qo_stride=(384, 192), ko_stride=(384, 192), dq_stride=(384, 192), dk_stride=(384, 192)), SCRATCH),
    # heads outermost, tokens of one buffer in turn
    (dict(dq=at(9), dk=at(9) + W), dict(nheads_q=2, dq_stride=(128, 2048), dk_stride=(128, 2048)), SCRATCH),
    # rows of different strides in one buffer: every second place of 64, then places of the other
    (dict(dq=at(9), dk=at(9) + W), dict(nheads_q=2, dq_stride=(384, 128), dk_stride=(512, 128)), SCRATCH),
    (dict(dq=at(9), dk=at(9) + 4 * W), dict(nheads_q=2, dq_stride=(384, 128), dk_stride=(512, 128)), ALIASING),
    (dict(dq=at(9), dk=at(9) + W // 2), dict(nheads_q=2, dq_stride=(384, 192), dk_stride=(384, 192)), ALIASING),
    (dict(dq=at(9), dk=at(9) + 2 * 384 * 2), dict(nheads_q=2, dq_stride=(384, 192), dk_stride=(384, 192)), ALIASING),
    (dict(dk=at(1) + W), dict(k_stride=(256, 128), dk_stride=(256, 128)), SCRATCH),
    (dict(dk=at(1) + W), dict(k_stride=(256, 64), dk_stride=(256, 64)), ALIASING),
    (dict(), dict(dq_stride=(64, 64)), ALIASING),
    (dict(), dict(dq_stride=(64, 1024)), SCRATCH),
])
def test_gradients_of_fused_buffers(ssd, ptrs, kw, status):
    assert scratch(ssd, ptrs, **kw) == status


@pytest.mark.gpu
@pytest.mark.parametrize("order", ["thcd", "tchd", "htcd", "cthd", "chtd", "hctd"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_in_a_fused_projection(order, dtype):
    # q, k, v of one buffer: tokens t, heads h and the three c in any order
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd
    T, H, D = 37, 4, 64
    size = dict(t=T, h=H, c=3, d=D)
    g = torch.Generator(device="cuda").manual_seed(2)
    buf, grad = (torch.randn([size[x] for x in order], device="cuda", generator=g).to(dtype) for _ in range(2))
    perm = [order.index(x) for x in "cthd"]
    q, k, v = buf.permute(perm)
    dq, dk, dv = grad.permute(perm)
    cos, sin = ssd.rope_table(64, D)
    tab = (torch.ones(D, device="cuda"), None, cos, sin, torch.arange(T, dtype=torch.int32, device="cuda"))
    c = lambda x: x.clone(memory_format=torch.contiguous_format)  # noqa: E731
    v0, dv0 = c(v), c(dv)
    want = ssd.qk_norm_rope_bwd(c(q), c(k), *tab, c(dq), c(dk))
    got = ssd.qk_norm_rope_bwd(q, k, *tab, dq, dk, dq=dq, dk=dk)
    qo, ko = ssd.qk_norm_rope_fwd(c(q), c(k), *tab)
    ssd.qk_norm_rope_fwd(q, k, *tab, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert torch.equal(dq, want["dq"]) and torch.equal(dk, want["dk"]) and torch.equal(dv, dv0)
    assert all(torch.equal(got[n], want[n]) for n in ("dq_weight", "dk_weight"))
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, v0)
