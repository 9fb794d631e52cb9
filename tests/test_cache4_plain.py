"""The format of a cache in 4 bits, by hand, and how near it comes."""
import numpy as np

import cache4_plain as c4


def test_bytes_by_hand():
    x = np.zeros((1, 1, 1, 16))
    x[..., :8] = [7, -7, 3, 2.5, 3.5, -0.5, 1.5, 0.25]
    cache, values = c4.cache_of(x)
    # scale 1 is byte 128; halves go to even numbers
    n = [7, -7, 3, 2, 4, 0, 2, 0]
    assert values.reshape(-1)[:8].tolist() == n
    c = [v + 8 for v in n]
    assert cache.reshape(-1).tolist() == [c[0] + 16 * c[2], c[4] + 16 * c[6], c[1] + 16 * c[3], c[5] + 16 * c[7]] + [0x88] * 4 + [128]


def test_scales():
    assert c4.SCALES[0] == 2.0 ** -16 and c4.SCALES[128] == 1 and c4.SCALES[254] == 57344 and c4.SCALES[131] == 1.375
    for most, byte in [(7, 128), (7 * 1.0625, 128), (7 * 1.1875, 130), (7 * 1.07, 129), (0, 0), (1e-9, 0), (1e9, 254), (np.inf, 255), (np.nan, 255)]:
        x = np.zeros((1, 16))
        x[0, 3] = most
        assert c4.quantise(x)[0][0, 0] == byte, most


def test_values_again():
    """Half a step off at most, values written back give the same bytes, bf16 holds them."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((4, 3, 8, 64)) * np.exp(rng.uniform(-8, 8, (4, 3, 8, 1)))
    cache, v = c4.cache_of(x)
    g = np.abs(x).reshape(4, 3, 8, 4, 16).max(-1, keepdims=True)
    # a step is a seventh of the largest, and up to 1/17 more or less by the scale's rounding
    assert (np.abs(v - x).reshape(4, 3, 8, 4, 16) <= g / 14 * 18 / 17).all()
    assert np.array_equal(c4.cache_of(v)[0], cache)
    assert np.array_equal(c4.values(cache, 8, 64), v)
    assert np.array_equal((v.astype(np.float32).view(np.uint32) & 0xffff), np.zeros(v.shape))
