"""Products of 8-bit integers in every form that the choice for 9 to 256 tokens knows: tiles of 32, 64 and 128 tokens; CTAs alone on
their SMs or with K in 1 to 8 ranges, one or two of them on an SM; no drain of the accumulators, one, and several.
The forms named beside the sizes are those of 152 SMs.  Bit for bit against sums in fp64, which hold them exactly."""
import pytest
import torch

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


ALONE = [  # M, N, K: no drain, one, two or three of each tile
    (28, 19456, 100), (28, 19133, 8919), (30, 17195, 16717),
    (40, 201, 333), (50, 13134, 4442), (40, 13114, 9377),
    (196, 300, 200), (177, 6108, 2062), (206, 5040, 4133), (128, 16384, 6300),
]
SHARED = [  # two CTAs on an SM; 1, 2, 3, 4, 6, 8 ranges of each tile
    (29, 19615, 1), (24, 12238, 2326), (12, 10835, 1314), (26, 6672, 2212), (14, 4927, 2946), (22, 3513, 3907),
    (52, 19478, 1), (64, 12320, 2624), (47, 10580, 1425), (49, 6652, 2470), (37, 5097, 3718), (50, 3736, 5162),
    (176, 9731, 1), (256, 10240, 640), (159, 5255, 1501), (128, 10576, 2560), (243, 3266, 2105), (190, 2456, 3154), (238, 1555, 4123),
]
APART = [  # one CTA on an SM: ranges without a drain, with one, with several
    (16, 6684, 759), (24, 1, 533), (15, 1, 450), (30, 1, 708), (24, 1, 962),
    (26, 9240, 13657), (30, 8776, 29408), (17, 5676, 18577), (22, 4609, 25507), (12, 3604, 32958), (30, 2642, 36599), (26, 1, 33176),
    (52, 7058, 577), (46, 1, 513), (55, 9305, 6525), (61, 9096, 8330), (37, 5944, 6671), (51, 4694, 12818), (44, 2642, 13438), (62, 1, 32924),
    (132, 3261, 321), (118, 1, 321), (240, 4611, 2102), (171, 3272, 4204), (205, 2934, 3101), (143, 2101, 4165), (163, 1155, 6180), (221, 1, 8201),
    (125, 1, 16385),
]


@pytest.mark.parametrize("M,N,K", ALONE + SHARED + APART)
def test_forms(ssd, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M)
    a, w = (torch.randint(-128, 128, s, generator=g, device="cuda", dtype=torch.int8) for s in ((M, K), (N, K)))
    sa, sw = torch.rand(M, generator=g, device="cuda") + 0.5, torch.rand(N, generator=g, device="cuda") + 0.5
    want = (a.double() @ w.double().t()).float() * sa[:, None] * sw
    packed = ssd.q8_pack_weight(w)
    for dtype in (BF, F):
        for _ in range(2):
            assert torch.equal(ssd.q8_matmul(a, sa, packed, sw, dtype=dtype), want.to(dtype))
    assert ssd.device_error() == 0
