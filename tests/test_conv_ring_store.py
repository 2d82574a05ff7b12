"""What a prompt leaves for the steps behind it: entries, padding, types and refusals (the same on the CPU and on the GPU)."""
import pytest
import torch

BF, F = torch.bfloat16, torch.float32
DEVICES = ["cpu", pytest.param("cuda", marks=pytest.mark.gpu)]


@pytest.fixture(scope="module")
def ssd():
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd as mod
    return mod


def make(dev, B, S, K, C, dtype, seed=1):
    if dev == "cuda" and not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator().manual_seed(seed)
    return torch.randn(S, K, C, generator=g).to(dev, dtype), torch.randn(B, K - 1, C, generator=g).to(dev, dtype)


def expected(ring, state, slots, lengths):
    ring, K = ring.clone(), ring.shape[1]
    for b, (s, n) in enumerate(zip(slots.tolist(), lengths.tolist())):
        if 0 <= s < ring.shape[0] and n >= 0:
            for j in range(K - 1):
                ring[s, (n - K + 1 + j) % K] = state[b, j]
    return ring


@pytest.mark.parametrize("dev", DEVICES)
@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
@pytest.mark.parametrize("K,dtype", [(2, F), (3, BF), (4, BF), (4, F)])
@pytest.mark.parametrize("slots,lengths", [
    ([3, 0, 5], [7, 1, 100]), ([2], [0]), ([1, -1, 4], [5, 6, 7]), ([-1, 6, 2 ** 31 - 1, 0], [1, 2, 3, 2]), ([6, -2], [3, 4]), ([1, 2], [-1, 9]),
    ([0, 5, -1], [2 ** 31 - 1, 2, 8]), ([], [])])
def test_entries_and_padding(ssd, slots, lengths, K, dtype, itype, dev):
    """Rows with a slot outside the pool (6 slots) or a negative length store nothing, in no slot."""
    ring, state = make(dev, len(slots), 6, K, 5, dtype)
    slots, lengths = torch.tensor(slots, dtype=itype, device=dev), torch.tensor(lengths, dtype=itype, device=dev)
    want = expected(ring, state, slots, lengths)
    assert ssd.conv_ring_store(ring, state, slots, lengths) is None
    assert torch.equal(ring, want)


@pytest.mark.parametrize("bad", [
    dict(ring=(6, 4)), dict(ring=(6, 1, 5)), dict(state=(2, 4, 5)), dict(state=(3, 3, 5)), dict(state=(2, 3, 6)), dict(slots=(3,)), dict(lengths=(1,)),
    dict(lengths=(2, 1))])
def test_wrong_shapes(ssd, bad):
    shape = dict(dict(ring=(6, 4, 5), state=(2, 3, 5), slots=(2,), lengths=(2,)), **bad)
    t = {k: torch.zeros(v, dtype=F if k in ("ring", "state") else torch.int64) for k, v in shape.items()}
    with pytest.raises(ValueError):
        ssd.conv_ring_store(t["ring"], t["state"], t["slots"], t["lengths"])


def test_wrong_types(ssd):
    ring, state = make("cpu", 2, 6, 4, 5, F)
    i = torch.zeros(2, dtype=torch.int64)
    for args in ((ring.half(), state.half(), i, i), (ring, state.bfloat16(), i, i), (ring, state, i.float(), i), (ring, state, i, i.to(torch.int16)),
                 (ring, state.to("meta"), i, i), (ring, state, i.to("meta"), i)):
        with pytest.raises(ValueError):
            ssd.conv_ring_store(*args)


@pytest.mark.gpu
def test_captured_and_on_another_stream(ssd):
    ring, state = make("cuda", 3, 6, 4, 40, BF)
    slots, lengths = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([1, -1, 3], [9, 5, 2]))
    want = expected(ring, state, slots, lengths)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = ring.clone()
    torch.cuda.synchronize()
    ssd.conv_ring_store(other, state, slots, lengths, stream=st)
    st.synchronize()
    assert torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssd.conv_ring_store(ring, state, slots, lengths)
    slots.copy_(torch.tensor([5, 2, 17], dtype=torch.int32))
    want = expected(ring, state, slots, lengths)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ring, want)
