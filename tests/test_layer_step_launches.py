"""The kernels around the scan start as programmatic dependents, as the attention layer's do: while the launch before them
still writes what they read.  The read-only load path asks for data that do not change while a kernel lives, so none of
them may use it."""
import glob
import os

import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_space_04_gb300", "csrc")


def test_no_read_only_loads():
    files = [f for name in ("ssd_norm*", "ssd_q8*", "ssd_step*") for f in glob.glob(os.path.join(CSRC, name))]
    assert len(files) >= 7
    for f in files:
        with open(f) as src:
            s = src.read()
        for word in ("__ldg(", "ld.global.nc", "ld.nc", "__restrict__", "tex1D"):
            assert word not in s, f"{word} in {os.path.basename(f)}"


def test_scales_read_ahead_of_the_wait_come_from_l2():
    """The product for 9 to 256 tokens reads its scales before it waits for the launch in front, when only L2 is sure to hold
    what the launches before that one wrote: an ordinary load may find an older line in L1."""
    with open(os.path.join(CSRC, "ssd_q8_mid.cu")) as f:
        s = f.read()
    assert s.count("__ldcg(p.as +") == 1 and s.count("__ldcg(p.ws +") == 1
    assert "p.as[" not in s and "p.ws[" not in s


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 8, 40, 300])
def test_products_directly_behind_the_norm(rows):
    """Norms and products in the same buffers again and again, each the one before's dependent: the bits of a waited-for sequence."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd
    D, N, steps = 1024, 1000, 40
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(steps, rows, D, device="cuda", generator=g)
    weight = torch.randn(steps, D, device="cuda", generator=g)
    packed = ssd.q8_pack_weight(torch.randint(-127, 128, (N, D), device="cuda", generator=g, dtype=torch.int8))
    sw = torch.rand(N, device="cuda", generator=g)
    h, w = torch.empty(rows, D, device="cuda"), torch.empty(D, device="cuda")
    q, scale = torch.empty(rows, D, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    ws = torch.empty(max(16, ssd.q8_matmul_workspace_size(q, N)), dtype=torch.uint8, device="cuda")

    def run(wait):
        outs = []
        for i in range(steps):
            ssd.add_rmsnorm_fwd(weight[i:i + 1], ones, out=w.view(1, D))   # (the next launch's weight)
            if wait:
                torch.cuda.synchronize()
            ssd.add_rmsnorm_fwd(x[i], w, out=h)
            if wait:
                torch.cuda.synchronize()
            ssd.add_rmsnorm_q8_fwd(h, w, q=q, scale=scale)
            if wait:
                torch.cuda.synchronize()
            outs.append(ssd.q8_matmul(q, scale, packed, sw, dtype=torch.float32, workspace=ws))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs

    ones = torch.ones(D, device="cuda")
    ref = run(True)
    for _ in range(3):
        assert all(torch.equal(a, b) and torch.isfinite(a).all() for a, b in zip(run(False), ref))
