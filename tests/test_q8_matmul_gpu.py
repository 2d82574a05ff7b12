"""GPU parity of the products of 8-bit integers.  The sums are exact, and what follows them is three roundings in a stated
order, so every result is compared bit for bit."""
import numpy as np
import pytest
import torch

from oracle import layer_step

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ssd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd as mod
    return mod


def ints(seed, *shape, lo=-127, hi=127):
    return torch.randint(lo, hi + 1, shape, generator=torch.Generator().manual_seed(seed), dtype=torch.int64).to(torch.int8).cuda()


def scales(seed, n):
    return torch.rand(n, generator=torch.Generator().manual_seed(seed)).cuda() + 0.5


def expected(acc, sa, sw, dtype):
    """float(sum) * a_scale * w_scale, each rounded to fp32, then to dtype."""
    y = acc.astype(np.float32) * sa.cpu().numpy()[:, None] * sw.cpu().numpy()[None, :]
    return torch.from_numpy(y).to(dtype)


def check(ssd, a, w, dtype, **kw):
    sa, sw = scales(3, a.shape[0]), scales(4, w.shape[0])
    y = ssd.q8_matmul(a, sa, ssd.q8_pack_weight(w), sw, dtype=dtype, **kw)
    assert torch.equal(y.cpu(), expected(layer_step.q8_matmul(a, w), sa, sw, dtype))


SIZES = [  # M, N, K
    (1, 1, 1), (1, 128, 64), (1, 300, 2560), (2, 129, 65), (7, 127, 63), (8, 1000, 129), (16, 256, 1024), (17, 384, 1040), (31, 200, 2048),
    (33, 640, 777), (64, 130, 4100), (65, 512, 512), (77, 333, 1001), (100, 64, 8192), (128, 1056, 640), (129, 257, 320), (200, 900, 1536),
    (255, 128, 192), (256, 256, 256), (257, 513, 1025), (500, 300, 2100), (1000, 700, 500), (1025, 257, 1100), (2048, 512, 768), (3000, 130, 130), (288, 20000, 70), (416, 9000, 100), (33000, 40, 64),
]


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(ssd, M, N, K, dtype):
    check(ssd, ints(1, M, K), ints(2, N, K), dtype)


@pytest.mark.parametrize("M", [1, 20, 130, 1100])
@pytest.mark.parametrize("K", [1024, 1040, 9000, 65536])
def test_largest_values(ssd, M, K):
    """All products of one sign and the largest there are: sums far past what fp32 holds exactly."""
    a, w = torch.full((M, K), -128, dtype=torch.int8, device="cuda"), torch.full((140, K), -128, dtype=torch.int8, device="cuda")
    a[M // 2] = 127
    w[5, ::3] = 127
    w[139, 1::2] = 0
    check(ssd, a, w, F)


@pytest.mark.parametrize("M", [1, 3, 40, 150, 1030])
def test_views(ssd, M):
    """Rows of any stride and alignment, in and out; what lies between the result's rows stays."""
    K, N = 333, 201
    a = ints(5, M, K + 46)[:, 13:13 + K]
    w = ints(6, N, K + 3)[:, 1:1 + K]
    sa, sw = scales(7, M), scales(8, N)
    for dtype in (BF, F):
        buf = torch.full((M, N + 9), 7.0, dtype=dtype, device="cuda")
        y = ssd.q8_matmul(a, sa, ssd.q8_pack_weight(w), sw, out=buf[:, 5:5 + N])
        assert torch.equal(y.cpu(), expected(layer_step.q8_matmul(a, w), sa, sw, dtype))
        assert (buf[:, :5] == 7).all() and (buf[:, 5 + N:] == 7).all()
    one = ssd.q8_matmul(a[:1].expand(M, K), sa, ssd.q8_pack_weight(w), sw, dtype=F)   # one row for all tokens
    assert torch.equal(one, ssd.q8_matmul(a[:1].expand(M, K).contiguous(), sa, ssd.q8_pack_weight(w), sw, dtype=F))


def test_packed_layout(ssd):
    N, K = 300, 150
    w = ints(9, N, K)
    full = torch.zeros(384, 192, dtype=torch.int8)
    full[:N, :K] = w.cpu()
    assert torch.equal(ssd.q8_pack_weight(w).cpu(), full.view(3, 128, 12, 16).transpose(1, 2).reshape(-1))


def test_a_row_does_not_depend_on_the_others(ssd):
    """The same token in batches of any size: the same bits."""
    N, K = 700, 2560
    a, packed, sw = ints(10, 1500, K), ssd.q8_pack_weight(ints(11, N, K)), scales(12, N)
    sa = scales(13, 1500)
    whole = ssd.q8_matmul(a, sa, packed, sw, dtype=F)
    for n in (1, 2, 9, 33, 100, 129, 300, 700, 1100):
        assert torch.equal(ssd.q8_matmul(a[-n:], sa[-n:], packed, sw, dtype=F), whole[-n:])


def test_scales_that_are_no_numbers(ssd):
    """A token with scale NaN (a norm's row that held one) gives NaN, and no other token does; scale 0 gives 0."""
    a, w = ints(14, 20, 256), ints(15, 130, 256)
    a[3] = 0
    sa, sw = scales(16, 20), scales(17, 130)
    sa[3], sa[4] = float("nan"), 0.0
    y = ssd.q8_matmul(a, sa, ssd.q8_pack_weight(w), sw)
    assert y[3].isnan().all() and not y[4].any()
    keep = torch.ones(20, dtype=torch.bool)
    keep[3] = False
    assert y[keep.cuda()].isfinite().all()


def test_no_tokens(ssd):
    y = ssd.q8_matmul(ints(18, 0, 64), scales(19, 0), ssd.q8_pack_weight(ints(20, 10, 64)), scales(21, 10))
    assert y.shape == (0, 10)


@pytest.mark.parametrize("M,N,K", [(3, 300, 700), (150, 300, 700), (1200, 300, 700)])
def test_own_workspace_and_stream(ssd, M, N, K):
    a, w, sa, sw = ints(22, M, K), ints(23, N, K), scales(24, M), scales(25, N)
    packed = ssd.q8_pack_weight(w)
    need = ssd.q8_matmul_workspace_size(a, N)
    ws = torch.full((need + 64,), 171, dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = ssd.q8_matmul(a, sa, packed, sw, workspace=ws[:need] if need else None, stream=st)
    st.synchronize()
    assert torch.equal(y.cpu(), expected(layer_step.q8_matmul(a, w), sa, sw, BF))
    assert (ws[need:] == 171).all()


def test_offsets_past_32_bits(ssd):
    """Rows of a and of the result whose offsets pass 2^32."""
    K, N, M = 200, 140, 3
    stride = (1 << 31) + 31
    big = torch.empty(2 * stride + K, dtype=torch.int8, device="cuda")
    a = big.as_strided((M, K), (stride, 1))
    a.copy_(ints(26, M, K))
    out = torch.empty(2 * stride + N, dtype=BF, device="cuda").as_strided((M, N), (stride, 1))
    w, sa, sw = ints(27, N, K), scales(28, M), scales(29, N)
    ssd.q8_matmul(a, sa, ssd.q8_pack_weight(w), sw, out=out)
    assert torch.equal(out.cpu(), expected(layer_step.q8_matmul(a, w), sa, sw, BF))
