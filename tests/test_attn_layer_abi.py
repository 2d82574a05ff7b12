"""CPU checks of the attention-layer entry points' argument validation: every
refusal happens before any CUDA call (the pointers here are made up)."""
import ctypes

import pytest

INVALID, NULL, MISALIGNED, UNSUPPORTED, ALIASING, DTYPE = 1, 2, 3, 4, 7, 9


@pytest.fixture(scope="module")
def ssd():
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd as mod
    return mod


def at(i):
    """Made-up arrays 1 GiB apart."""
    return (i + 1) << 30


PLAN = ("lens", "new_lens", "block_table", "free_ring", "ring_pos", "lens_out", "granted", "start", "positions", "token_req",
        "slots", "ring_pos_out", "counts")


def plan(ssd, ptrs=None, **kw):
    base = dict(nreq=10, max_tokens=64, ring_size=100, page_size=16, max_pages=8, flags=0, reserved=0)
    base.update(kw)
    d = ssd.SsdPlanDims(*(base[f] for f, _ in ssd.SsdPlanDims._fields_))
    p = {n: at(i) for i, n in enumerate(PLAN)}
    p.update(ptrs or {})
    return ssd.lib().ssd_paged_plan(*(p[n] for n in PLAN), d, None)


@pytest.mark.parametrize("kw,ptrs,status", [
    (dict(nreq=-1), {}, INVALID), (dict(max_tokens=-1), {}, INVALID), (dict(max_tokens=2 ** 31), {}, INVALID),
    (dict(ring_size=0), {}, INVALID), (dict(page_size=0), {}, INVALID), (dict(max_pages=0), {}, INVALID),
    (dict(page_size=2 ** 16, max_pages=2 ** 15), {}, INVALID), (dict(flags=1), {}, INVALID), (dict(reserved=1), {}, INVALID),
    (dict(nreq=8193), {}, UNSUPPORTED),
    *[({}, {n: None}, NULL) for n in PLAN],
    *[({}, {n: at(i) + 8}, MISALIGNED) for i, n in enumerate(PLAN)],
    ({}, dict(granted=at(0)), ALIASING), ({}, dict(slots=at(2)), ALIASING), ({}, dict(lens_out=at(0) + 16), ALIASING),
    ({}, dict(free_ring=at(2) + 64), ALIASING), ({}, dict(counts=at(4)), ALIASING),
])
def test_plan_refusals(ssd, kw, ptrs, status):
    assert plan(ssd, ptrs, **kw) == status


def test_plan_null_dims(ssd):
    assert ssd.lib().ssd_paged_plan(*[at(i) for i in range(13)], None, None) == NULL


QK = ("q", "k", "v", "q_weight", "k_weight", "cos", "sin", "positions", "q_out", "k_out", "k_cache", "v_cache", "slots")


def qk_dims(ssd, **kw):
    base = dict(ntokens=16, max_pos=64, npages=4, nheads_q=4, nheads_k=2, headdim=64, rotary_dim=64, page_size=8, dtype=1, flags=0,
                eps=1e-6, q_stride=(256, 64), k_stride=(128, 64), v_stride=(128, 64), qo_stride=(256, 64), ko_stride=(128, 64),
                dq_stride=(256, 64), dk_stride=(128, 64), kc_stride=(1024, 128, 64), vc_stride=(1024, 128, 64))
    base.update(kw)
    return ssd.SsdQkDims(*(base[f] for f, _ in ssd.SsdQkDims._fields_))


def qk(ssd, ptrs=None, **kw):
    p = {n: at(i) for i, n in enumerate(QK)}
    p.update(ptrs or {})
    return ssd.lib().ssd_qk_norm_rope_fwd(*(p[n] for n in QK), qk_dims(ssd, **kw), None)


QK_DIMS = [
    (dict(ntokens=-1), INVALID), (dict(ntokens=2 ** 31), INVALID), (dict(max_pos=-1), INVALID), (dict(nheads_q=0), INVALID),
    (dict(nheads_k=0), INVALID), (dict(headdim=0), INVALID), (dict(rotary_dim=-16), INVALID), (dict(rotary_dim=80), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(flags=2), INVALID), (dict(dtype=2), DTYPE),
    (dict(headdim=60, rotary_dim=16), UNSUPPORTED), (dict(headdim=264), UNSUPPORTED), (dict(rotary_dim=24), UNSUPPORTED),
    (dict(q_stride=(260, 64)), MISALIGNED), (dict(ko_stride=(128, 68)), MISALIGNED), (dict(k_stride=(-128, 64)), INVALID),
    (dict(q_stride=(2 ** 61, 64)), INVALID),
]


@pytest.mark.parametrize("kw,status", QK_DIMS + [
    (dict(page_size=0), INVALID), (dict(npages=-1), INVALID), (dict(kc_stride=(1024, 130, 64)), MISALIGNED),
    (dict(vc_stride=(2 ** 60, 128, 64)), INVALID)])
def test_qk_dims_refusals(ssd, kw, status):
    assert qk(ssd, **kw) == status


@pytest.mark.parametrize("ptrs,status", [
    *[({n: None}, NULL) for n in ("q", "k", "v", "cos", "sin", "positions", "q_out", "k_cache", "v_cache", "slots")],
    *[({n: at(i) + 4}, MISALIGNED) for i, n in enumerate(QK) if n != "positions"],
    (dict(positions=at(7) + 2), MISALIGNED),
    (dict(q_out=at(1)), ALIASING), (dict(k_out=at(0)), ALIASING), (dict(q_out=at(3)), ALIASING), (dict(k_cache=at(2)), ALIASING),
    (dict(v_cache=at(8)), ALIASING), (dict(k_out=at(8) + 64), ALIASING), (dict(k_cache=at(12)), ALIASING),
])
def test_qk_pointer_refusals(ssd, ptrs, status):
    assert qk(ssd, ptrs) == status


def test_qk_without_a_cache_needs_k_out(ssd):
    assert qk(ssd, dict(k_cache=None, v_cache=None, slots=None, k_out=None)) == NULL


def test_qk_views_of_one_buffer_are_told_apart(ssd):
    # q, k, v are views of one [16, 8, 64] buffer; k_out over v (an input, with a cache) or half over k overlaps
    s = (512, 64)
    kw = dict(q_stride=s, k_stride=s, v_stride=s, ko_stride=s)
    p = dict(q=at(0), k=at(0) + 512, v=at(0) + 768)
    assert qk(ssd, dict(p, k_out=at(0) + 768), **kw) == ALIASING
    assert qk(ssd, dict(p, k_out=at(0) + 512 - 128), **kw) == ALIASING
    # output rows that share memory
    assert qk(ssd, qo_stride=(256, 0)) == ALIASING


BWD = ("q", "k", "q_weight", "k_weight", "cos", "sin", "positions", "dq_out", "dk_out", "dq", "dk", "dq_weight", "dk_weight")


def bwd(ssd, ptrs=None, ws=(None, 0), **kw):
    p = {n: at(i) for i, n in enumerate(BWD)}
    p.update(ptrs or {})
    return ssd.lib().ssd_qk_norm_rope_bwd(*(p[n] for n in BWD), *ws, qk_dims(ssd, **kw), None)


@pytest.mark.parametrize("kw,status", QK_DIMS + [(dict(dq_stride=(256, 60)), MISALIGNED)])
def test_bwd_dims_refusals(ssd, kw, status):
    assert bwd(ssd, **kw) == status


@pytest.mark.parametrize("ptrs,status", [
    *[({n: None}, NULL) for n in ("q", "k", "cos", "sin", "positions", "dq_out", "dk_out", "dq", "dk")],
    *[({n: at(i) + 4}, MISALIGNED) for i, n in enumerate(BWD) if n != "positions"],
    (dict(dq=at(0)), ALIASING), (dict(dk=at(7)), ALIASING), (dict(dq_weight=at(2)), ALIASING), (dict(dk_weight=at(11)), ALIASING),
    (dict(dq=at(10)), ALIASING),
])
def test_bwd_pointer_refusals(ssd, ptrs, status):
    assert bwd(ssd, ptrs) == status


def test_bwd_workspace_refusals(ssd):
    n = ctypes.c_uint64(0)
    assert ssd.lib().ssd_qk_norm_rope_bwd_workspace_size(qk_dims(ssd), ctypes.byref(n)) == 0 and n.value > 0
    assert ssd.lib().ssd_qk_norm_rope_bwd_workspace_size(qk_dims(ssd), None) == NULL
    assert bwd(ssd, ws=(at(20), n.value - 1)) == 8
    assert bwd(ssd, ws=(at(20) + 8, n.value)) == MISALIGNED
    assert bwd(ssd, ws=(at(0), n.value)) == ALIASING


ATTN = ("q", "k_cache", "v_cache", "block_table", "positions", "start", "out", "lse")


def attn_dims(ssd, **kw):
    base = dict(nrows=16, nreq=4, npages=32, nheads=8, nkv=2, headdim=64, page_size=16, max_pages=8, window=0, dtype=1, flags=0,
                scale=0.125, reserved=0, q_stride=(512, 64), o_stride=(512, 64), kc_stride=(2048, 128, 64),
                vc_stride=(2048, 128, 64), table_stride=8)
    base.update(kw)
    return ssd.SsdAttnDims(*(base[f] for f, _ in ssd.SsdAttnDims._fields_))


def attn(ssd, ptrs=None, ws=(None, 0), **kw):
    p = {n: at(i) for i, n in enumerate(ATTN)}
    p.update(ptrs or {})
    return ssd.lib().ssd_paged_attn_fwd(*(p[n] for n in ATTN), *ws, attn_dims(ssd, **kw), None)


@pytest.mark.parametrize("kw,status", [
    (dict(nrows=-1), INVALID), (dict(nreq=-1), INVALID), (dict(npages=-1), INVALID), (dict(nheads=0), INVALID),
    (dict(nkv=3), INVALID), (dict(nkv=0), INVALID), (dict(headdim=0), INVALID), (dict(page_size=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(page_size=2 ** 16, max_pages=2 ** 15), INVALID), (dict(window=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(flags=1), INVALID), (dict(reserved=1), INVALID), (dict(table_stride=-1), INVALID),
    (dict(dtype=5), DTYPE), (dict(headdim=60), UNSUPPORTED), (dict(headdim=264), UNSUPPORTED), (dict(nreq=16385), UNSUPPORTED),
    (dict(q_stride=(512, 60)), MISALIGNED), (dict(kc_stride=(2044, 128, 64)), MISALIGNED), (dict(o_stride=(2 ** 60, 64)), INVALID),
    (dict(o_stride=(0, 64)), ALIASING),
])
def test_attn_dims_refusals(ssd, kw, status):
    assert attn(ssd, **kw) == status


@pytest.mark.parametrize("ptrs,status", [
    *[({n: None}, NULL) for n in ("q", "k_cache", "v_cache", "block_table", "positions", "out")],
    *[({n: at(i) + 2}, MISALIGNED) for i, n in enumerate(ATTN)],
    (dict(out=at(0) + 128), ALIASING), (dict(out=at(1)), ALIASING), (dict(lse=at(3)), ALIASING), (dict(lse=at(6)), ALIASING),
    (dict(lse=at(0)), ALIASING),
])
def test_attn_pointer_refusals(ssd, ptrs, status):
    assert attn(ssd, ptrs) == status


@pytest.mark.parametrize("name", ["kc_stride", "vc_stride"])
def test_attn_page_and_token_strides_have_a_limit(ssd, name):
    big = 2 ** 35   # bf16: 2^32 times 16 bytes
    assert attn(ssd, **{name: (big, 128, 64)}) == UNSUPPORTED
    assert attn(ssd, **{name: (128, big, 64)}) == UNSUPPORTED


def test_qk_rows_have_a_limit(ssd):
    assert qk(ssd, ntokens=2 ** 30 // 4, nheads_q=8) == UNSUPPORTED


def test_attn_rows_without_start_are_requests(ssd):
    assert attn(ssd, dict(start=None)) == INVALID
