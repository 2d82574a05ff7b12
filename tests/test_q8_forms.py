"""CPU restatements of the arithmetic that the 8-bit kernels rely on being exact."""
import numpy as np


def test_widening_to_half_is_exact():
    """Byte b with its sign bit turned, below the bits of 1024.0, is 1024 + 128 + b; 1152 off that is b."""
    b = np.arange(-128, 128).astype(np.int8)
    bits = (0x6400 | (b.view(np.uint8) ^ 0x80).astype(np.uint16)).astype(np.uint16)
    assert np.array_equal(bits.view(np.float16) - np.float16(1152.0), b.astype(np.float16))


def test_sums_of_1024_products_are_exact_in_fp32():
    """No partial sum of 1024 products of 8-bit integers leaves the whole numbers that fp32 holds, in any order."""
    assert 128 * 128 * 1024 <= 2 ** 24
    rng = np.random.default_rng(0)
    a = rng.integers(-128, 128, (50, 1024))
    w = rng.integers(-128, 128, (50, 1024))
    a[0], w[0] = -128, -128
    a[1], w[1] = -128, 127
    for x, y in zip(a, w):
        acc = np.float32(0)
        for p in (x * y).astype(np.float32):
            acc += p
        assert int(acc) == int((x * y).sum())


def test_rounding_by_the_large_constant():
    """The lowest byte of 1.5 2^23 + x is x to the nearest whole number, even ones at halves."""
    x = np.concatenate([np.arange(-127, 127.01, 0.125), np.random.default_rng(1).uniform(-127, 127, 10000)]).astype(np.float32)
    bits = (x.astype(np.float64) + 12582912.0).astype(np.float32).view(np.uint32)
    assert np.array_equal((bits & 0xff).astype(np.uint8).view(np.int8), np.rint(x).astype(np.int8))


def test_transposing_eight_lanes():
    """Three exchanges of pairs turn 8 lanes' columns of 16-bit values into rows, as the results of many tokens are stored."""
    v = np.random.default_rng(2).integers(0, 1 << 16, (8, 8))   # [lane][row]
    p = v[:, 0::2] | v[:, 1::2] << 16
    lane = np.arange(8)
    h4, h2, h1 = (lane & 4) > 0, (lane & 2) > 0, (lane & 1) > 0
    s = [np.where(h4, p[:, i], p[:, i + 2])[lane ^ 4] for i in (0, 1)]
    a = [np.where(h4, s[0], p[:, 0]), np.where(h4, s[1], p[:, 1]), np.where(h4, p[:, 2], s[0]), np.where(h4, p[:, 3], s[1])]
    s = [np.where(h2, a[0], a[1])[lane ^ 2], np.where(h2, a[2], a[3])[lane ^ 2]]
    b = [np.where(h2, s[0], a[0]), np.where(h2, a[1], s[0]), np.where(h2, s[1], a[2]), np.where(h2, a[3], s[1])]
    out = np.zeros((8, 8), dtype=np.int64)
    for c in range(4):
        o = b[c][lane ^ 1]
        out[:, 2 * c] = np.where(h1, o >> 16, b[c] & 0xffff)
        out[:, 2 * c + 1] = np.where(h1, b[c] >> 16, o & 0xffff)
    assert np.array_equal(out, v.T)


def test_ring_of_inputs():
    """Entry t mod K holds the input of position t: after each step the K - 1 before the next are there, and the one that
    is overwritten is the one that no tap reads."""
    for K in (2, 3, 4):
        ring = [None] * K
        for t in range(20):
            for j in range(1, min(K - 1, t) + 1):
                assert ring[(t - j) % K] == t - j and (t - j) % K != t % K
            ring[t % K] = t
