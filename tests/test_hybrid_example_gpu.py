"""The hybrid serving example end to end: requests that join and leave, token by
token, against the same sequences taken in one step each by a fresh server.
Both run the same arithmetic in another split (other shares, other steps), so in
fp32 the logits agree to the rounding of a few layers: 2^-12 of their size."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_04_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("hybrid_decode", os.path.join(ROOT, "examples", "hybrid_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["hybrid_decode"] = mod
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("window", [0, 20])
def test_steps_agree_with_whole_sequences(ex, window):
    c = ex.Config(dtype=torch.float32, window=window, page_size=8)
    w = ex.make_weights(c, 3)
    g = torch.Generator().manual_seed(4)
    lens = [5, 40, 1, 23]
    seqs = [torch.randint(c.vocab, (n + 6,), generator=g).tolist() for n in lens]
    server = ex.Server(c, w, 4, pages=40)
    # prompts in one step, the second request a step later; then one token each
    got = {}
    first = {i: seqs[i][:lens[i]] for i in (0, 2, 3)}
    server.step(first)
    work = {i: [seqs[i][lens[i]]] for i in (0, 2, 3)}
    work[1] = seqs[1][:lens[1] + 1]
    server.step(work)
    for k in range(1, 6):
        got = server.step({i: [seqs[i][lens[i] + k]] for i in range(4)})
    for i in range(4):
        ref = ex.Server(c, w, 1, pages=40).step({0: seqs[i]})[0]
        assert (got[i] - ref).abs().max() <= 2.0 ** -12 * ref.abs().max()


def test_pages_come_back_and_requests_are_independent(ex):
    c = ex.Config(dtype=torch.float32, page_size=8, max_len=64)
    w = ex.make_weights(c, 5)
    g = torch.Generator().manual_seed(6)
    prompts = [torch.randint(c.vocab, (n,), generator=g).tolist() for n in (9, 30, 4, 17, 25, 8)]
    # two slots and pages for little more than two requests: all others wait for pages given back
    out, _ = ex.generate(c, w, prompts, 5, slots=2, pages=11)
    for p, o in zip(prompts, out):
        alone, _ = ex.generate(c, w, [p], 5, slots=1, pages=8)
        assert o == alone[0] and len(o) == len(p) + 5


def test_bf16_runs(ex):
    c = ex.Config()
    out, steps = ex.generate(c, ex.make_weights(c), [[1, 2, 3], [4] * 50, [7]], 4, slots=2, pages=64)
    assert [len(o) for o in out] == [7, 54, 5] and steps >= 8
