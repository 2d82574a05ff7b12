"""The attention layer's calls work on the thread's current device: tensors, a stream
or a workspace of another one are refused, before anything is launched or allocated,
for remembered layouts too.  CPU: the devices, and tensors on them, are stand-ins."""
import pytest
import torch

I32, I64, BF = torch.int32, torch.int64, torch.bfloat16


class Fake:
    """What the wrappers ask of a tensor."""

    def __init__(self, *shape, dtype=BF, device="cuda:1"):
        self.like = torch.empty(*shape, dtype=dtype, device="meta")
        self.device, self.dtype, self.shape, self.is_cuda = torch.device(device), dtype, self.like.shape, True
        for name in ("stride", "dim", "is_contiguous", "numel", "element_size"):
            setattr(self, name, getattr(self.like, name))

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return 1 << 30

    def __getitem__(self, at):
        raise AssertionError("not asked for")


class FakeStream:
    def __init__(self, index):
        self.device_index, self.cuda_stream = index, 7


def calls(ssd, dev, **kw):
    t = lambda *s, dtype=BF: Fake(*s, dtype=dtype, device=dev)  # noqa: E731
    i = lambda *s: t(*s, dtype=I32)  # noqa: E731
    f = lambda *s: t(*s, dtype=torch.float32)  # noqa: E731
    out = dict(lens=i(4), granted=i(4), start=i(5), positions=i(8), token_req=i(8), slots=t(8, dtype=I64),
               ring_pos=t(2, dtype=I64), counts=i(4))
    yield lambda: ssd.paged_plan(i(4), i(4), i(4, 6), i(30), t(2, dtype=I64), page_size=16, max_tokens=8, out=out, **kw)
    qk = (t(8, 4, 64), t(8, 2, 64), f(64), None, f(32, 32), f(32, 32), i(8))
    yield lambda: ssd.qk_norm_rope_fwd(*qk, q_out=t(8, 4, 64), k_out=t(8, 2, 64), **kw)
    yield lambda: ssd.qk_norm_rope_bwd(*qk, t(8, 4, 64), t(8, 2, 64), dq=t(8, 4, 64), dk=t(8, 2, 64), **kw)
    yield lambda: ssd.paged_attn_fwd(t(8, 4, 64), t(9, 16, 2, 64), t(9, 16, 2, 64), i(8, 6), i(8), out=t(8, 4, 64), lse=f(8, 4), **kw)


@pytest.fixture
def ssd(monkeypatch):
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd as mod

    class NoLibrary:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was reached")

    monkeypatch.setattr(mod, "_lib", NoLibrary())
    monkeypatch.setattr(mod, "_known", {})
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: empty(*a, device="meta", **k))
    return mod


def test_tensors_of_another_device(ssd):
    for _ in range(2):   # the second time with remembered layouts
        for call in calls(ssd, "cuda:1"):
            with pytest.raises(ValueError, match="current device"):
                call()


def test_a_stream_of_another_device(ssd):
    for _ in range(2):
        for call in calls(ssd, "cuda:0", stream=FakeStream(1)):
            with pytest.raises(ValueError, match="stream"):
                call()


def test_a_workspace_of_another_device(ssd):
    for kind, call in enumerate(calls(ssd, "cuda:0", workspace=Fake(1 << 20, dtype=torch.uint8))):
        if kind >= 2:   # (the others take none)
            with pytest.raises(ValueError, match="workspace"):
                call()


def test_the_current_device_passes(ssd):
    for call in calls(ssd, "cuda:0", stream=FakeStream(0)):
        with pytest.raises((AssertionError, AttributeError), match="ssd_|data_ptr"):   # (the library is reached)
            call()
