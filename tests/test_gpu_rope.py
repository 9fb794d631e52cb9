"""rope_store against norm and rotation in 64 bits; what is copied, bit for bit.

Tolerances, with u = 2^-24 and (a, b) a pair before its rotation, after the norm:
* the norm: the sum of D squares is off by (D / 2 + 8) u at most in any order of its
  additions here (at most D / 2 of them follow one another), its root by half of that,
  1 / sqrt by 2 u, the two products by u each: (D / 4 + 8) u of the element;
* sine and cosine: the angle's fraction of a turn is rounded to 24 bits, 2 pi 2^-25 at
  most, the functions to two units of their last place, 2 u: 5.2 u of |a| + |b|, the
  product and the sum 2 u more;
* bf16: the result is rounded once, 2^-8 of it.
"""
import math

import pytest
import torch

import speculative_decoding_drafter_markov_gb300 as dsp
from speculative_decoding_drafter_markov_gb300 import _lib
from test_gpu_target import err_word, ints, shifted

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]
EPS = 1e-6


def freqs(rot, base=1e6):
    return torch.pow(torch.tensor(base, dtype=torch.float64), -torch.arange(0, rot, 2).double() / max(rot, 1)).float().cuda()


def expect(x, pos, freq, weight, interleaved, eps=EPS):
    """(values, sizes |a| + |b| of each element's pair) in 64 bits."""
    x = x.double()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    half = freq.shape[0]
    rot = 2 * half
    angle = pos.double()[:, None] * freq.double()
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, half), slice(half, rot))
    a, b = x[..., first], x[..., second]
    out, size = x.clone(), x.abs()
    out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    size[..., first] = size[..., second] = a.abs() + b.abs()
    return out, size


def near(got, want, size, D, norm):
    u = 2.0 ** -24
    tol = (8 + (D / 4 + 8 if norm else 0)) * u * size
    if got.dtype == torch.bfloat16:
        tol = tol * 1.01 + 2.0 ** -8 * want.abs()
    off = (got.double() - want).abs()
    assert (off <= tol).all(), float((off / tol.clamp(min=1e-300)).max())


def case(N, Hq, H, D, rot, dtype, seed=0, odd=0, page=16, far=200000):
    g = torch.Generator(device="cuda").manual_seed(seed)
    fused = torch.randn((N, Hq + 2 * H + (1 if odd else 0), D + odd), generator=g, device="cuda").to(dtype)
    fused = fused[:, (1 if odd else 0):, :D]
    pos = torch.randint(0, far, (N,), generator=g, device="cuda", dtype=torch.int32)
    pages = N // page + 2
    slot = torch.randperm(pages * page, generator=g, device="cuda")[:N].int()
    w = lambda: (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dtype)  # noqa: E731
    caches = [torch.randn((pages, H, page, D), generator=g, device="cuda").to(dtype) for _ in range(2)] if H else None
    return dict(q=fused[:, :Hq], k=fused[:, Hq:Hq + H], v=fused[:, Hq + H:], pos=pos, slot=slot, freq=freqs(rot), wq=w(), wk=w(), caches=caches,
                page=page)


def check(s, interleaved=False, norm=True, cached=True, **kw):
    D = s["q"].shape[-1]
    err = err_word()
    weights = dict(q_weight=s["wq"], k_weight=s["wk"]) if norm else {}
    q_want, q_size = expect(s["q"], s["pos"], s["freq"], weights.get("q_weight"), interleaved)
    k_want, k_size = expect(s["k"], s["pos"], s["freq"], weights.get("k_weight"), interleaved)
    q0, k0, v0 = (s[n].clone() for n in "qkv")
    if cached:
        kc, vc = (c.clone() for c in s["caches"])
        out = dsp.rope_store(s["q"], s["k"], s["v"], s["pos"], s["freq"], eps=EPS, interleaved=interleaved, slot=s["slot"], k_cache=kc, v_cache=vc,
                             err=err, **weights, **kw)
        assert set(out) == {"q"}
        page, off = s["slot"].long() // s["page"], s["slot"].long() % s["page"]
        near(kc[page, :, off], k_want, k_size, D, norm)
        assert torch.equal(vc[page, :, off], v0)
        for c, before in zip((kc, vc), s["caches"]):  # and nothing else
            c[page, :, off] = before[page, :, off]
            assert torch.equal(c, before)
    else:
        out = dsp.rope_store(s["q"], s["k"], None, s["pos"], s["freq"], eps=EPS, interleaved=interleaved, err=err, **weights, **kw)
        near(out["k"], k_want, k_size, D, norm)
        rest = slice(2 * s["freq"].shape[0], D)
        if not norm:
            assert torch.equal(out["k"][..., rest], k0[..., rest])
    near(out["q"], q_want, q_size, D, norm)
    assert int(err) == 0
    if "out" not in kw:
        assert torch.equal(s["q"], q0) and torch.equal(s["k"], k0)
    return out


SIZES = [(1, 32, 8, 128, 128), (9, 8, 2, 64, 64), (33, 4, 4, 80, 40), (65, 7, 1, 96, 48), (5, 3, 3, 256, 256), (40, 16, 2, 128, 64),
         (17, 2, 1, 80, 80), (11, 2, 2, 24, 16), (6, 4, 2, 72, 36), (8, 3, 1, 7, 6), (4, 1, 1, 2, 2), (3, 2, 1, 1, 0), (50, 6, 3, 128, 0),
         (2500, 8, 2, 128, 128), (9, 4, 4, 256, 100), (12, 5, 2, 200, 200), (3, 64, 8, 192, 64), (6, 2, 2, 16, 16), (6, 2, 2, 8, 8)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("N,Hq,H,D,rot", SIZES)
def test_sizes(dtype, interleaved, norm, N, Hq, H, D, rot):
    s = case(N, Hq, H, D, rot, dtype, seed=N + D)
    check(s, interleaved, norm, cached=True)
    check(s, interleaved, norm, cached=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("odd", [1, 4, 2])
def test_views(dtype, odd):
    for D, rot in ((128, 128), (64, 32)):
        check(case(21, 4, 2, D, rot, dtype, seed=odd, odd=odd), cached=True)
        check(case(21, 4, 2, D, rot, dtype, seed=odd, odd=odd), cached=False, interleaved=True)


@pytest.mark.parametrize("dtype", TYPES)
def test_far_positions(dtype):
    s = case(10, 2, 2, 128, 128, dtype)
    s["pos"] = ints([0, 1, -1, 131071, 1 << 20, (1 << 24) + 1, 2 ** 31 - 1, -2 ** 31, 12345678, -99999])
    check(s, cached=False)
    check(s, cached=True, interleaved=True, norm=False)
    # frequencies above one turn, tiny and none
    s["freq"][:8] = torch.tensor([6.5, 100.0, 30000.0, 1e-20, 0.0, 1e-40, -1.0, -0.37])
    s["pos"] = ints([0, 1, -1, 3, 17, 131071, 1 << 20, 5, 99, -99999])
    check(s, cached=False)


@pytest.mark.parametrize("dtype", TYPES)
def test_queries_or_keys_alone(dtype):
    s = case(9, 4, 2, 64, 64, dtype)
    both = dsp.rope_store(s["q"], s["k"], None, s["pos"], s["freq"], q_weight=s["wq"], k_weight=s["wk"])
    assert torch.equal(dsp.rope_store(s["q"], None, None, s["pos"], s["freq"], q_weight=s["wq"])["q"], both["q"])
    only = dsp.rope_store(None, s["k"], None, s["pos"], s["freq"], k_weight=s["wk"])
    assert set(only) == {"k"} and torch.equal(only["k"], both["k"])
    kc, vc = s["caches"]
    assert dsp.rope_store(None, s["k"], s["v"], s["pos"], s["freq"], k_weight=s["wk"], slot=s["slot"], k_cache=kc, v_cache=vc) == {}
    page, off = s["slot"].long() // s["page"], s["slot"].long() % s["page"]
    assert torch.equal(kc[page, :, off], both["k"]) and torch.equal(vc[page, :, off], s["v"])
    # a norm of one of the two
    one = dsp.rope_store(s["q"], s["k"], None, s["pos"], s["freq"], q_weight=s["wq"])
    assert torch.equal(one["q"], both["q"]) and torch.equal(one["k"], dsp.rope_store(None, s["k"], None, s["pos"], s["freq"])["k"])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_in_place_and_into_views(dtype, odd, interleaved, norm):
    s = case(70, 8, 2, 128, 96, dtype, odd=odd)
    weights = dict(q_weight=s["wq"], k_weight=s["wk"]) if norm else {}
    kw = dict(interleaved=interleaved, **weights)
    want = dsp.rope_store(s["q"], s["k"], None, s["pos"], s["freq"], **kw)
    wide = torch.full((70, 12, 136), 7.0, dtype=dtype, device="cuda")
    views = {"q": wide[:, :8, :128], "k": wide[:, 9:11, :128]}
    assert dsp.rope_store(s["q"], s["k"], None, s["pos"], s["freq"], out=views, **kw) is views
    assert torch.equal(views["q"], want["q"]) and torch.equal(views["k"], want["k"])
    assert (wide[:, 8] == 7).all() and (wide[:, 11] == 7).all() and (wide[:, :, 128:] == 7).all()
    v = s["v"].clone()
    dsp.rope_store(s["q"], s["k"], None, s["pos"], s["freq"], out={"q": s["q"], "k": s["k"]}, **kw)
    assert torch.equal(s["q"], want["q"]) and torch.equal(s["k"], want["k"]) and torch.equal(s["v"], v)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [128, 9])
def test_skipped_rows_and_bad_slots(dtype, D):
    s = case(6, 4, 2, D, 8, dtype)
    kc, vc = (c.clone() for c in s["caches"])
    last = kc.shape[0] * 16
    slot = ints([-1, 3, last, -5, last - 1, 0])
    out = {"q": torch.full((6, 4, D), 7.0, dtype=dtype, device="cuda")}
    err = err_word()
    dsp.rope_store(s["q"], s["k"], s["v"], s["pos"], s["freq"], slot=slot, k_cache=kc, v_cache=vc, out=out, err=err)
    assert int(err) == _lib.ERR_RANGE
    want = dsp.rope_store(s["q"], s["k"], None, s["pos"], s["freq"])
    keep, at = [1, 4, 5], [3, last - 1, 0]
    assert torch.equal(out["q"][keep], want["q"][keep]) and (out["q"][[0, 2, 3]] == 7).all()
    k_want, v_want = (c.clone() for c in s["caches"])
    for i, a in zip(keep, at):
        k_want[a // 16, :, a % 16], v_want[a // 16, :, a % 16] = want["k"][i], s["v"][i]
    assert torch.equal(kc, k_want) and torch.equal(vc, v_want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [128, 9])
def test_sizes_of_numbers(dtype, D):
    """Squares beyond 32 bits, heads of zeros, tiny ones; infinities and NaN stay in their head
    (and, unnormed, in their pair)."""
    rot = 8
    s = case(5, 2, 2, D, rot, dtype)
    x = s["q"].clone()
    x[0] *= 1e25
    x[1] = 0
    x[2] *= 1e-25
    big = dsp.rope_store(x, None, None, s["pos"], s["freq"], q_weight=s["wq"], eps=EPS)["q"]
    near(big, *expect(x, s["pos"], s["freq"], s["wq"], False), D, True)
    small = dsp.rope_store(x, None, None, s["pos"], s["freq"], q_weight=s["wq"], eps=1e-30)["q"]
    rows = [0, 3, 4]
    near(small[rows], *expect(x[rows], s["pos"][rows], s["freq"], s["wq"], False, 1e-30), D, True)
    assert not small[1].any() and torch.isfinite(small).all()
    for bad in (float("inf"), float("nan")):
        x = s["q"].clone()
        x[3, 1, 1] = bad
        want = dsp.rope_store(s["q"], None, None, s["pos"], s["freq"], q_weight=s["wq"])["q"]
        got = dsp.rope_store(x, None, None, s["pos"], s["freq"], q_weight=s["wq"])["q"]
        assert got[3, 1].isnan().any()
        want[3, 1] = got[3, 1] = 0
        assert torch.equal(got, want)
        want = dsp.rope_store(s["q"], None, None, s["pos"], s["freq"])["q"]
        got = dsp.rope_store(x, None, None, s["pos"], s["freq"])["q"]
        assert not torch.isfinite(got[3, 1, [1, 1 + rot // 2]]).any()
        want[3, 1, [1, 1 + rot // 2]] = got[3, 1, [1, 1 + rot // 2]] = 0
        assert torch.equal(got, want)


def test_offsets_beyond_32_bits():
    H, page, D = 8, 64, 128
    n_pages = (1 << 31) // (H * page * D) + 3
    s = case(3, 2, H, D, D, torch.bfloat16)
    kc, vc = (torch.zeros((n_pages, H, page, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slot = [n_pages * page - 1, n_pages * page - 64, 5]
    dsp.rope_store(s["q"], s["k"], s["v"], s["pos"], s["freq"], slot=ints(slot), k_cache=kc, v_cache=vc)
    k = dsp.rope_store(None, s["k"], None, s["pos"], s["freq"])["k"]
    assert torch.equal(kc[-1, :, -1], k[0]) and torch.equal(kc[-1, :, 0], k[1]) and torch.equal(kc[0, :, 5], k[2])
    assert torch.equal(vc[-1, :, -1], s["v"][0]) and int(torch.count_nonzero(kc[1:-1])) == 0


def test_in_a_graph_and_on_another_stream():
    s = case(40, 8, 2, 128, 128, torch.bfloat16)
    kw = dict(q_weight=s["wq"], k_weight=s["wk"], slot=s["slot"])
    want_c = [c.clone() for c in s["caches"]]
    want = dsp.rope_store(s["q"], s["k"], s["v"], s["pos"], s["freq"], k_cache=want_c[0], v_cache=want_c[1], **kw)["q"]
    a, b = ([c.clone() for c in s["caches"]] for _ in range(2))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = dsp.rope_store(s["q"], s["k"], s["v"], s["pos"], s["freq"], k_cache=a[0], v_cache=a[1], stream=side, **kw)["q"]
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(a[0], want_c[0]) and torch.equal(a[1], want_c[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dsp.rope_store(s["q"], s["k"], s["v"], s["pos"], s["freq"], k_cache=b[0], v_cache=b[1], **kw)["q"]
    pos = s["pos"].clone()
    for change in (7, 0):  # positions are read on the GPU
        s["pos"].copy_(pos + change)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(b[0], want_c[0]) and torch.equal(b[1], want_c[1])


def test_refusals():
    s = case(5, 4, 2, 64, 64, torch.bfloat16)
    q, k, v, pos, freq, slot, (kc, vc) = (s[n] for n in ("q", "k", "v", "pos", "freq", "slot", "caches"))
    cache = dict(slot=slot, k_cache=kc, v_cache=vc)
    for args, kw in [((None, None, None, pos, freq), {}), ((q, k, v[:, :1], pos, freq), cache), ((q, k, v, pos[:-1], freq), cache),
                     ((q, None, v, pos, freq), cache), ((q, k, v, pos, freq), dict(cache, slot=slot[:-1])),
                     ((q, k, v, pos, freq), dict(cache, v_cache=vc[1:])), ((q, k, v, pos, freq), dict(cache, k_cache=kc[:, :1])),
                     ((q, k, v, pos, freq), dict(k_cache=kc, v_cache=vc)), ((q.transpose(1, 2), k, v, pos, freq), {}),
                     ((q, k[:, :, :32], v, pos, freq), {}), ((q, k, v, pos, freq.cpu()), {}), ((q, k, v, pos, freq), dict(q_weight=s["wq"][:5])),
                     ((q, k, v, pos, freq), dict(out={"q": q[:, :1], "k": k}))]:
        with pytest.raises(ValueError):
            dsp.rope_store(*args, **kw)
    for args, kw in [((q, k.float(), None, pos, freq), {}), ((q, k, None, pos.long(), freq), {}), ((q, k, None, pos, freq.double()), {}),
                     ((q, k, None, pos, freq), dict(q_weight=s["wq"].float())), ((q.half(), None, None, pos, freq), {}),
                     ((q, k, None, pos, freq), dict(cache)), ((q, k, None, pos, freq), dict(out=[q, k]))]:
        with pytest.raises(TypeError):
            dsp.rope_store(*args, **kw)
    with pytest.raises(KeyError):
        dsp.rope_store(q, k, None, pos, freq, out={"q": q.clone()})
    for args, kw in [((q, k, None, pos, freqs(66)), {}), ((q, k, None, pos, freq), dict(q_weight=s["wq"], eps=0.0)),
                     ((q, k, None, pos, freq), dict(k_weight=s["wk"], eps=math.nan)),
                     ((torch.zeros((1, 1, 300), dtype=torch.bfloat16, device="cuda"), None, None, pos[:1], freq), {})]:
        with pytest.raises(dsp.DSparkError):
            dsp.rope_store(*args, **kw)
    assert dsp.rope_store(q[:0], k[:0], None, pos[:0], freq)["k"].shape == (0, 2, 64)
