"""A decode step's step plan, norm and rotary into the cache, and attention, captured
once in a CUDA graph and replayed while the requests grow: every replay gives the
bits of the same calls made one by one."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd as mod
    return mod


def state(dtype, R, ps, H, hk, D):
    g = torch.Generator().manual_seed(3)
    pages, dev = 40, "cuda"
    s = dict(lens=torch.zeros(R, dtype=torch.int32), table=torch.full((R, 8), -1, dtype=torch.int32),
             ring=torch.randperm(pages, generator=g).int(), ring_pos=torch.tensor([0, pages]),
             kc=torch.zeros(pages, ps, hk, D, dtype=dtype), vc=torch.zeros(pages, ps, hk, D, dtype=dtype))
    s = {k: v.to(dev) for k, v in s.items()}
    i32 = dict(dtype=torch.int32, device=dev)
    s["plan"] = dict(lens=s["lens"], granted=torch.empty(R, **i32), start=torch.empty(R + 1, **i32), positions=torch.empty(R, **i32),
                     token_req=torch.empty(R, **i32), slots=torch.empty(R, dtype=torch.int64, device=dev),
                     ring_pos=s["ring_pos"], counts=torch.empty(4, **i32))
    return s


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("own_workspace", [True, False])
def test_replays_equal_single_calls(ssd, dtype, own_workspace):
    R, ps, H, hk, D = 5, 8, 8, 2, 64
    cos, sin = ssd.rope_table(64, D)
    w = torch.linspace(0.5, 1.5, D, device="cuda")
    a, b = state(dtype, R, ps, H, hk, D), state(dtype, R, ps, H, hk, D)
    new = torch.ones(R, dtype=torch.int32, device="cuda")
    x = torch.zeros(R, H + 2 * hk, D, dtype=dtype, device="cuda")
    ws = None
    if own_workspace:
        n = ssd.paged_attn_workspace_size(x[:, :H], a["kc"], a["vc"], a["table"])
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def step(s):
        plan = ssd.paged_plan(s["lens"], new, s["table"], s["ring"], s["ring_pos"], page_size=ps, max_tokens=R,
                              out=s["plan"])
        q, k, v = x.split((H, hk, hk), dim=1)
        q, _ = ssd.qk_norm_rope_fwd(q, k, w, w, cos, sin, plan["positions"], v=v, k_cache=s["kc"], v_cache=s["vc"],
                                    slots=plan["slots"], return_k=False)
        return ssd.paged_attn_fwd(q, s["kc"], s["vc"], s["table"], plan["positions"], plan["start"], workspace=ws)

    step(state(dtype, R, ps, H, hk, D))   # (the library's first call outside of a capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step(a)
    g = torch.Generator().manual_seed(9)
    for i in range(20):
        x.copy_(torch.randn(x.shape, generator=g))
        new.copy_(torch.tensor([1, 1, i % 2, 1 if i > 4 else 0, -1 if i == 10 else 1]))
        graph.replay()
        ro, rl = step(b)
        torch.cuda.synchronize()
        assert torch.equal(out, ro) and torch.equal(lse, rl) and torch.isfinite(ro).all()
        assert all(torch.equal(a[k], b[k]) for k in a if k != "plan")
        assert all(torch.equal(a["plan"][k], b["plan"][k]) for k in b["plan"])
