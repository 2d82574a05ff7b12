"""The operators around the scan together, as a served layer uses them: against the fp64 oracles, captured and replayed,
on several streams, and in the serving example.

The chain's tolerance: 8-bit rows are off by half a step of 1/127 of a row's largest value at two places, the
projections' bf16 results by 2^-8, and everything behind them follows; what is compared are sums over hundreds of
such values, so 3 of 127 steps of the largest output.
"""
import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

from oracle import layer_step

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd as mod
    return mod


@pytest.fixture(scope="module")
def ex(ssd):
    spec = importlib.util.spec_from_file_location("hybrid_decode_m", os.path.join(ROOT, "examples", "hybrid_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    sys.modules["hybrid_decode_m"] = mod
    spec.loader.exec_module(mod)
    return mod


class Layer:
    """Weights, states and one step of a layer, in the given types."""

    def __init__(self, ssd, seed, rows, dtype, H=4, P=32, N=64, G=2, K=4, d=160):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
        self.ssd, self.dtype, self.dims = ssd, dtype, (H, P, N, G, K, d)
        self.inner, self.C = H * P, H * P + 2 * G * N
        self.norm, self.gate = 1 + 0.2 * r(d), 1 + 0.2 * r(self.inner)
        self.w_in, self.s_in = self.quantized(r(self.inner + self.C + H, d) / d ** 0.5)
        self.w_out, self.s_out = self.quantized(r(d, self.inner) / self.inner ** 0.5)
        self.p_in, self.p_out = ssd.q8_pack_weight(self.w_in), ssd.q8_pack_weight(self.w_out)
        self.cw, self.cb = r(self.C, K) / K, 0.1 * r(self.C)
        self.dt_bias, self.A_log, self.D = r(H) - 2, 0.3 * r(H), r(H)
        self.ring, self.states = r(rows + 2, K, self.C).to(dtype), r(rows + 2, H, P, N)
        self.slots = torch.randperm(rows + 2, generator=g)[:rows].int().cuda()
        self.pos = torch.randint(1, 50, (rows,), generator=g).int().cuda()
        self.x, self.res = r(rows, d).to(dtype), r(rows, d)

    @staticmethod
    def quantized(w):
        s = w.abs().amax(1) / 127
        return torch.clamp(torch.round(w / s[:, None]), -127, 127).to(torch.int8), s

    def step(self, **kw):
        ssd, (H, P, N, G, K, d) = self.ssd, self.dims
        q, s, res = ssd.add_rmsnorm_q8_fwd(self.x, self.norm, self.res, **kw)
        proj = ssd.q8_matmul(q, s, self.p_in, self.s_in, dtype=self.dtype, **kw)
        z, xbc, dt = proj[:, :self.inner], proj[:, self.inner:self.inner + self.C], proj[:, self.inner + self.C:]
        y = ssd.conv_scan_step(xbc, self.ring, self.cw, self.cb, dt, self.dt_bias, self.A_log, self.D, self.states, self.slots, self.pos,
                               ngroups=G, **kw)
        q, s = ssd.gated_rmsnorm_q8_fwd(y.view(-1, self.inner), z, self.gate, **kw)
        return ssd.q8_matmul(q, s, self.p_out, self.s_out, dtype=self.dtype, **kw), res

    def oracle(self):
        H, P, N, G, K, d = self.dims
        n = lambda t: t.double().cpu().numpy()  # noqa: E731
        v, h = layer_step.add_rmsnorm(self.x, self.norm, self.res, 1e-6)
        proj = v @ (n(self.w_in) * n(self.s_in)[:, None]).T
        z, xbc, dt = proj[:, :self.inner], proj[:, self.inner:self.inner + self.C], proj[:, self.inner + self.C:]
        y, _, states, _ = layer_step.conv_scan_step(xbc, self.ring, self.cw, self.cb, dt, self.dt_bias, self.A_log, self.D, self.states,
                                                    self.slots, self.pos, G)
        v, _ = layer_step.add_rmsnorm(y.reshape(-1, self.inner), self.gate, None, 1e-6, gate=z)
        return v @ (n(self.w_out) * n(self.s_out)[:, None]).T, h, states


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("rows", [1, 7, 40, 300])
def test_a_step_against_the_oracles(ssd, rows, dtype):
    layer = Layer(ssd, rows, rows, dtype)
    out, res, states = layer.oracle()
    got, gres = layer.step()
    assert np.abs(got.double().cpu().numpy() - out).max() <= 3 / 127 * np.abs(out).max()
    assert np.abs(gres.double().cpu().numpy() - res).max() <= 2.0 ** -22 * np.abs(res).max()
    assert np.abs(layer.states.double().cpu().numpy() - states).max() <= 3 / 127 * np.abs(states).max()


@pytest.mark.parametrize("rows", [2, 40, 300])
def test_replays_equal_single_calls(ssd, rows):
    a, b = Layer(ssd, 5, rows, BF), Layer(ssd, 5, rows, BF)
    Layer(ssd, 6, rows, BF).step()   # (the library's first call outside of a capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, res = a.step()
    g = torch.Generator().manual_seed(7)
    for _ in range(6):
        x = torch.randn(a.x.shape, generator=g).to(BF)
        a.x.copy_(x)
        b.x.copy_(x)
        a.pos += 1
        b.pos += 1
        graph.replay()
        ro, rr = b.step()
        torch.cuda.synchronize()
        assert torch.equal(out, ro) and torch.equal(res, rr) and torch.isfinite(ro.float()).all()
        assert torch.equal(a.states, b.states) and torch.equal(a.ring, b.ring)


def test_captured_gradients(ssd):
    n, D = 300, 1000
    g = torch.Generator().manual_seed(8)
    h, w, d, dr = (torch.randn(*s, generator=g).cuda() for s in ((n, D), (D,), (n, D), (n, D)))
    ssd.add_rmsnorm_bwd(h, w, d, dr)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx, dw = ssd.add_rmsnorm_bwd(h, w, d, dr)
    for _ in range(3):
        d.copy_(torch.randn(n, D, generator=g))
        graph.replay()
        rx, rw = ssd.add_rmsnorm_bwd(h, w, d, dr)
        torch.cuda.synchronize()
        assert torch.equal(dx, rx) and torch.equal(dw, rw)


def test_layers_on_streams_of_their_own(ssd):
    """Several layers at once, back to back on their own streams, give what they give alone."""
    sizes = [1, 8, 9, 40, 130, 300, 1]
    alone = [Layer(ssd, 20 + i, n, BF) for i, n in enumerate(sizes)]
    want = []
    for layer in alone:
        for _ in range(4):
            out = layer.step()
            layer.pos += 1
        torch.cuda.synchronize()
        want.append(out)
    layers = [Layer(ssd, 20 + i, n, BF) for i, n in enumerate(sizes)]
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    got = [None] * len(sizes)
    for k in range(4):
        for i, (layer, st) in enumerate(zip(layers, streams)):
            with torch.cuda.stream(st):
                got[i] = layer.step()
                layer.pos += 1
    torch.cuda.synchronize()
    for layer, ref, (o, r), (wo, wr) in zip(layers, alone, got, want):
        assert torch.equal(o, wo) and torch.equal(r, wr) and torch.equal(layer.states, ref.states) and torch.equal(layer.ring, ref.ring)
    assert ssd.device_error() == 0


def test_many_products_back_to_back(ssd):
    """Calls of every size one after another on one stream, each the other's dependent, without a wait between."""
    g = torch.Generator().manual_seed(9)
    i8 = lambda *s: torch.randint(-127, 128, s, generator=g).to(torch.int8).cuda()  # noqa: E731
    N, K = 1400, 1500
    packed, sw = ssd.q8_pack_weight(i8(N, K)), torch.rand(N, generator=g).cuda()
    cases = [(i8(m, K), torch.rand(m, generator=g).cuda()) for m in (1, 128, 8, 9, 600, 64, 256, 1200, 16, 257, 3, 200)]
    want = []
    for a, sa in cases:
        want.append(ssd.q8_matmul(a, sa, packed, sw))
        torch.cuda.synchronize()
    for _ in range(5):
        got = [ssd.q8_matmul(a, sa, packed, sw) for a, sa in cases]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert ssd.device_error() == 0


def test_example_requests_are_independent(ex):
    """8-bit layers served with continuous batching: each request's tokens are those that it gets alone."""
    c = ex.Config(layers="mm", page_size=8, max_len=64)
    w = ex.make_weights(c, 5)
    g = torch.Generator().manual_seed(6)
    prompts = [torch.randint(c.vocab, (n,), generator=g).tolist() for n in (9, 30, 1, 17, 2, 8)]
    out, _ = ex.generate(c, w, prompts, 5, slots=3, pages=24)
    for p, o in zip(prompts, out):
        alone, _ = ex.generate(c, w, [p], 5, slots=1, pages=8)
        assert o == alone[0] and len(o) == len(p) + 5


@pytest.mark.parametrize("dtype", [BF, F])
def test_example_steps_agree_with_whole_sequences(ex, dtype):
    """Tokens one by one, in twos and as a prompt: the logits differ by what 8-bit rows and bf16 rounding turn over."""
    c = ex.Config(layers="ma", dtype=dtype, page_size=8)
    w = ex.make_weights(c, 3)
    g = torch.Generator().manual_seed(4)
    seq = torch.randint(c.vocab, (30,), generator=g).tolist()
    server = ex.Server(c, w, 2, pages=40)
    server.step({1: seq[:20]})
    server.step({1: seq[20:21]})
    server.step({1: seq[21:26]})
    for t in seq[26:]:
        got = server.step({1: [t]})[1]
    ref = ex.Server(c, w, 1, pages=40).step({0: seq})[0]
    assert (got - ref).abs().max() <= 3 / 127 * ref.abs().max()
