"""The attention layer's kernels start as programmatic dependents: while the launch
before them still writes what they read.  The read-only load path asks for data
that do not change while a kernel lives, so none of them may use it."""
import glob
import os

import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_space_04_gb300", "csrc")


def test_no_read_only_loads():
    files = glob.glob(os.path.join(CSRC, "ssd_paged_*")) + glob.glob(os.path.join(CSRC, "ssd_qk_*"))
    assert len(files) >= 7
    for f in files:
        with open(f) as src:
            s = src.read()
        for word in ("__ldg(", "ld.global.nc", "ld.nc", "__restrict__", "tex1D"):
            assert word not in s, f"{word} in {os.path.basename(f)}"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("in_place", [False, True])
def test_attention_directly_behind_the_plan(dtype, in_place):
    # pages of one token: every step's newest table entries are written by the launch directly in front
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd
    R, steps, H, hk, D = 300, 40, 4, 2, 64
    pages = R * (steps + 1)
    g = torch.Generator(device="cuda").manual_seed(5)
    kc, vc = (torch.randn(pages, 1, hk, D, device="cuda", generator=g).to(dtype) for _ in range(2))
    q = torch.randn(R, H, D, device="cuda", generator=g).to(dtype)
    new = torch.ones(R, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    ring = torch.randperm(pages, device="cuda", generator=g).int()

    def serve(wait):
        lens, table = torch.zeros(R, **i32), torch.full((R, steps + 1), -1, **i32)
        free, pos, outs = ring.clone(), torch.tensor([0, pages], device="cuda"), []
        kept = dict(granted=torch.empty(R, **i32), start=torch.empty(R + 1, **i32), positions=torch.empty(R, **i32),
                    token_req=torch.empty(R, **i32), slots=torch.empty(R, dtype=torch.int64, device="cuda"), counts=torch.empty(4, **i32))
        for _ in range(steps):
            out = dict(kept, lens=lens, ring_pos=pos) if in_place else None
            plan = ssd.paged_plan(lens, new, table, free, pos, page_size=1, max_tokens=R, out=out)
            lens, pos = plan["lens"], plan["ring_pos"]
            if wait:
                torch.cuda.synchronize()
            outs.append(ssd.paged_attn_fwd(q, kc, vc, table, plan["positions"], plan["start"]))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs

    ref = serve(True)
    for _ in range(3):
        for (a, al), (b, bl) in zip(serve(False), ref):
            assert torch.equal(a, b) and torch.equal(al, bl) and torch.isfinite(a).all()
