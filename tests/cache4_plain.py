"""A cache in 4 bits by its definition, in numpy and 64 bits: what the tests of
cache_store4 and tree_attention4 compare with."""
import numpy as np

PLACES = [(0, 2), (4, 6), (1, 3), (5, 7)]  # the elements of each byte of eight, low half first
SCALES = np.array([2.0 ** (b // 8 - 16) * (1 + (b % 8) / 8) for b in range(255)] + [np.nan])


def quantise(x):
    """(bytes, codes n) of x [.., D]: scale bytes [.., D / 16], whole numbers [.., D]."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 16)
    most = np.abs(g).max(-1)
    fine = np.isfinite(g).all(-1)
    a = np.where(fine, most, 1.0) / 7
    b = np.clip(np.searchsorted(SCALES[:255], a, side="right") - 1, 0, 253)
    lo, hi = SCALES[b], SCALES[b + 1]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (b % 2 == 1))
    b = np.where(fine, b + up, 255)
    n = np.clip(np.rint(np.where(fine[..., None], g, 0) / np.where(fine, SCALES[b], 1)[..., None]), -7, 7)
    return b.astype(np.uint8), n.reshape(x.shape).astype(int)


def held(b, n):
    """The values that bytes and codes stand for."""
    return (n.reshape(*b.shape, 16) * SCALES[b][..., None]).reshape(n.shape)


def pack(n):
    """Code bytes [.., D / 2]."""
    c = (n + 8).reshape(*n.shape[:-1], -1, 8)
    return np.stack([c[..., i] | c[..., j] << 4 for i, j in PLACES], -1).astype(np.uint8).reshape(*n.shape[:-1], -1)


def cache_of(x):
    """[pages, H, page D 9 / 16] bytes of a cache [pages, H, page, D], and the values held."""
    b, n = quantise(x)
    flat = x.shape[:2] + (-1,)
    return np.concatenate([pack(n).reshape(flat), b.reshape(flat)], -1), held(b, n)


def values(cache, page, D):
    """What a cache [pages, H, page D 9 / 16] of bytes stands for: [pages, H, page, D]."""
    codes = cache[..., :page * D // 2].reshape(*cache.shape[:2], page, D // 8, 4)
    n = np.zeros(codes.shape[:-1] + (8,), int)
    for byte, (i, j) in enumerate(PLACES):
        n[..., i], n[..., j] = (codes[..., byte] & 15).astype(int) - 8, (codes[..., byte] >> 4).astype(int) - 8
    b = cache[..., page * D // 2:].reshape(*cache.shape[:2], page, D // 16)
    return held(b, n.reshape(*cache.shape[:2], page, D))
