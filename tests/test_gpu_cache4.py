"""cache_store4 against the format's definition: bytes and values are equal, whatever
the inputs, since both roundings are exact."""
import numpy as np
import pytest
import torch

import cache4_plain as c4
import speculative_decoding_drafter_markov_gb300 as dsp
from speculative_decoding_drafter_markov_gb300 import _lib
from test_gpu_target import err_word, ints, shifted

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]


def write(cache, page, D, slot, x):
    """The rows x [N, H, D] into numpy cache bytes, one after the other; the values held [N, H, D]."""
    b, n = c4.quantise(x.double().cpu().numpy())
    codes = c4.pack(n)
    for i, s in enumerate(slot):
        if 0 <= s < cache.shape[0] * page:
            pg, off = s // page, s % page
            cache[pg, :, off * D // 2:(off + 1) * D // 2] = codes[i]
            cache[pg, :, page * D // 2 + off * D // 16:page * D // 2 + (off + 1) * D // 16] = b[i]
    return c4.held(b, n)


def check(k, v, slot, page, seed=0, **kw):
    N, H, D = k.shape
    g = torch.Generator(device="cuda").manual_seed(seed)
    n_pages = max(max(slot, default=0) // page + 1, 2)
    caches = [torch.randint(0, 256, (n_pages, H, page * D * 9 // 16), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
    want = [c.cpu().numpy() for c in caches]
    values = [write(w, page, D, slot, x) for w, x in zip(want, (k, v))]
    err = err_word()
    plain = [c.clone() for c in caches]
    assert dsp.cache_store4(k, v, ints(slot), *plain, err=err) is None
    out = dsp.cache_store4(k, v, ints(slot), *caches, values=True, err=err, **kw)
    assert int(err) == 0
    keep = np.array(slot) >= 0
    for c, p, w, name, x in zip(caches, plain, want, "kv", values):
        assert np.array_equal(c.cpu().numpy(), w) and torch.equal(c, p)
        assert out[name].dtype == k.dtype
        assert np.array_equal(out[name].double().cpu().numpy()[keep], x[keep], equal_nan=True)


def rows(N, H, D, dtype, seed, views=False):
    """Keys and values, normal with sizes over many powers of two, out of a fused projection."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    fused = torch.randn((N, 2 * H + 1, D + (3 if views else 0)), generator=g, device="cuda")
    fused = (fused * torch.exp(4 * torch.randn((N, 2 * H + 1, 1), generator=g, device="cuda"))).to(dtype)
    return fused[:, :H, :D], fused[:, H:2 * H, :D]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("views", [False, True])
@pytest.mark.parametrize("N,H,D,page", [(1, 1, 16, 8), (1, 8, 128, 16), (7, 3, 48, 8), (33, 8, 128, 16), (300, 2, 80, 24), (5, 1, 256, 1),
                                        (700, 4, 64, 64), (3000, 8, 128, 32)])
def test_bytes(dtype, views, N, H, D, page):
    k, v = rows(N, H, D, dtype, N + D, views)
    slot = np.random.default_rng(N).permutation((N // page + 2) * page)[:N]
    slot[N // 2] = -1 if N > 1 else slot[0]
    check(k, v, slot.tolist(), page)


@pytest.mark.parametrize("dtype", TYPES)
def test_halves_and_edges(dtype):
    """Quotients halfway between two whole numbers and maxima halfway between two scales, at
    every scale; values just beside them in 32 bits; zeros, tiny and huge ones."""
    scale = c4.SCALES[:255]
    middle = (scale[1:] + scale[:-1]) / 2
    groups = []
    for most in np.concatenate([scale, middle, [1e-12, 2.0 ** -18, 57344 * 1.03, 1e30]]):
        s = scale[min(c4.quantise(np.array([[7 * most] + [0.0] * 15]))[0][0, 0], 254)]
        half = [(i + 0.5) * s for i in range(7)]
        groups.append([7 * most] + half + [-h for h in half] + [0.0])
    x = np.array(groups)
    near = [x]
    if dtype == torch.float32:
        f = x.astype(np.float32)
        near += [np.nextafter(f, np.float32(np.inf)), np.nextafter(f, np.float32(-np.inf))]
    x = np.concatenate(near)
    x = np.concatenate([x, np.zeros((-len(x) % 8, 16))]).reshape(-1, 1, 128)
    k = torch.from_numpy(x).to(dtype).cuda()
    check(k, -k, list(range(len(x))), 16)


def test_every_bf16_number_beside_every_fraction():
    """Each bf16 magnitude of eight bits against each of the eight fractions of a scale."""
    x = []
    for m in range(8):
        s = 1 + m / 8
        for e in range(-4, 4):
            v = 2.0 ** e * (1 + np.arange(128) / 128)
            v = v[v <= 7 * s]
            for i in range(0, len(v), 15):
                part = v[i:i + 15]
                x.append([7 * s] + part.tolist() + [0.0] * (15 - len(part)))
    x = np.array(x)
    x = np.concatenate([x, np.zeros((-len(x) % 8, 16))]).reshape(-1, 1, 128)
    k = torch.from_numpy(x).to(torch.bfloat16).cuda()
    assert np.array_equal(k.double().cpu().numpy(), x)
    check(k, -k, list(range(len(x))), 16)


@pytest.mark.parametrize("dtype", TYPES)
def test_infinities_and_nan(dtype):
    k, v = (x.clone() for x in rows(6, 2, 64, dtype, 1))
    k[0, 0, 5], k[1, 1, 63], k[2, 0, 16], v[3, 1, 0], v[3, 1, 33] = float("nan"), float("inf"), -float("inf"), float("nan"), float("inf")
    k[5, 0] = float("nan")
    check(k, v, [3, 40, 11, 5, 70, 16], 16)


@pytest.mark.parametrize("dtype", TYPES)
def test_addresses(dtype):
    """Rows that do not start on 16 bytes, heads before rows, one row for all."""
    k, v = rows(20, 4, 64, dtype, 2)
    slot = list(range(1, 21))
    check(shifted(k), v, slot, 16)
    check(k, shifted(v), slot, 16)
    first = lambda x: x.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    check(first(k), first(v), slot, 16)
    check(k[:1].expand(20, -1, -1), v[:, :1].expand(-1, 4, -1), slot, 16)


def test_skipped_rows_and_bad_slots():
    k, v = rows(5, 2, 64, torch.bfloat16, 3)
    caches = [dsp.cache4(3, 2, 16, 64) for _ in range(2)]
    out = {n: torch.full((5, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for n in "kv"}
    err = err_word()
    slot = [-1, 3, 48, -7, 47]
    assert dsp.cache_store4(k, v, ints(slot), *caches, out=out, err=err) is out
    assert int(err) == _lib.ERR_RANGE
    for c, x, n in zip(caches, (k, v), "kv"):
        want = np.zeros(c.shape, np.uint8)
        values = write(want, 16, 64, slot, x)
        assert np.array_equal(c.cpu().numpy(), want)
        assert (out[n][[0, 2, 3]] == 7).all()
        assert np.array_equal(out[n][[1, 4]].double().cpu().numpy(), values[[1, 4]])


def test_offsets_beyond_32_bits():
    H, page, D = 8, 64, 128
    n_pages = (1 << 32) // (H * page * D * 9 // 16) + 3
    k, v = rows(3, H, D, torch.bfloat16, 4)
    slot = [n_pages * page - 1, n_pages * page - 64, 5]
    caches = [dsp.cache4(n_pages, H, page, D) for _ in range(2)]
    assert caches[0].numel() > 1 << 32
    out = dsp.cache_store4(k, v, ints(slot), *caches, values=True)
    for c, x, n in zip(caches, (k, v), "kv"):
        last = np.zeros((1,) + tuple(c.shape[1:]), np.uint8)
        values = write(last, page, D, [63, 0, -1], x)
        assert np.array_equal(c[-1:].cpu().numpy(), last)
        assert np.array_equal(out[n].double().cpu().numpy(), values)
        assert not c[1:-1].any()


def test_in_a_graph_and_on_another_stream():
    k, v = rows(40, 4, 64, torch.bfloat16, 5)
    slot = ints(list(range(40)))
    want = [dsp.cache4(4, 4, 16, 64) for _ in range(2)]
    dsp.cache_store4(k, v, slot, *want)
    a, b = ([dsp.cache4(4, 4, 16, 64) for _ in range(2)] for _ in range(2))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    dsp.cache_store4(k, v, slot, *a, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsp.cache_store4(k, v, slot, *b)
    for _ in range(2):
        b[0].zero_(), b[1].zero_()
        graph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(a[i], want[i]) and torch.equal(b[i], want[i])


def test_refusals():
    k, v = rows(5, 2, 64, torch.bfloat16, 6)
    kc, vc = (dsp.cache4(3, 2, 16, 64) for _ in range(2))
    slot = ints([0, 1, 2, 3, 4])
    with pytest.raises(ValueError):
        dsp.cache4(3, 2, 16, 72)
    with pytest.raises(ValueError):
        dsp.cache4(3, 2, 1, 64)
    for bad in [(k, v[:, :1], slot, kc, vc), (k, v, slot[:-1], kc, vc), (k, v, slot, kc, vc[1:]), (k, v, slot, kc, vc[:, :, 16:]),
                (k, v, slot, kc[:, :, 1:], vc), (k[:, :, :40], v[:, :, :40], slot, kc, vc), (k, v, slot, kc.cpu(), vc),
                (k[..., ::2], v[..., ::2], slot, kc, vc), (k[:, 0], v[:, 0], slot, kc, vc), (k, v, slot, kc.view(3, 2, 4, -1), vc)]:
        with pytest.raises(ValueError):
            dsp.cache_store4(*bad)
    for bad in [(k, v.float(), slot, kc, vc), (k, v, slot.long(), kc, vc), (k.half(), v.half(), slot, kc, vc),
                (k, v, slot, kc.view(torch.int8), vc)]:
        with pytest.raises(TypeError):
            dsp.cache_store4(*bad)
    with pytest.raises(KeyError):
        dsp.cache_store4(k, v, slot, kc, vc, out={"k": torch.empty_like(k)})
    off = torch.empty(kc.numel() + 8, dtype=torch.uint8, device="cuda")[8:].view(kc.shape)
    with pytest.raises(dsp.DSparkError, match="aligned"):
        dsp.cache_store4(k, v, slot, off, vc)
    with pytest.raises(dsp.DSparkError, match="aligned"):
        dsp.cache_store4(k, v, slot, kc, vc, out={"k": shifted(k), "v": torch.empty_like(v).contiguous()})
    assert dsp.cache_store4(k[:0], v[:0], slot[:0], kc, vc, values=True)["k"].shape == (0, 2, 64)
