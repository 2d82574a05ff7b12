"""The 8-bit product's scratch is what the header says, on the CPU."""
import ctypes
import random

import pytest


@pytest.fixture(scope="module")
def ssd():
    from selective_state_space_04_gb300 import build
    build.build()
    from selective_state_space_04_gb300 import ssd as mod
    return mod


def stated(M, N, K):
    up = lambda a, b: -(-a // b)  # noqa: E731
    if M <= 8:
        return 0
    if M <= 256:
        return 128 * up(M, 128) * 128 * up(K, 64)
    return 16384 * up(K, 64) * (up(N, 128) + up(min(M, 32768), 128)) + 32768


def test_scratch(ssd):
    r = random.Random(3)
    sizes = [(m, 300, 500) for m in (0, 1, 8, 9, 128, 129, 256, 257, 32768, 32769, 2 ** 31 - 1)]
    sizes += [tuple(int(2 ** r.uniform(0, e)) for e in (18, 24, 16)) for _ in range(500)]
    for M, N, K in sizes:
        n = ctypes.c_uint64(0)
        d = ssd.SsdQ8Dims(M, N, K, 0, 0, K, N)
        assert ssd.lib().ssd_q8_matmul_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0
        assert n.value == stated(M, N, K), (M, N, K)
