"""Norms of heads whose squares are beyond fp32, up to its largest numbers, in both of rope_store's
kernels (heads in pieces of 8 or 16 bytes, and any size).  Tolerances as in test_gpu_rope."""
import pytest
import torch

import speculative_decoding_drafter_markov_gb300 as dsp
from test_gpu_rope import EPS, TYPES, case, expect, near

pytestmark = pytest.mark.gpu
LAYOUTS = [(128, 128), (128, 32), (64, 64), (256, 256), (80, 40), (9, 8), (7, 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", LAYOUTS)
def test_all_of_a_head_is_large(dtype, interleaved, D, rot):
    """Every element between 2^e and 2^(e + 1), of either sign: D squares of 2^252 are beyond
    fp32 after any factor above 2^-66 too."""
    powers = [60, 63, 64, 96, 120, 124, 125, 126, 127]
    s = case(len(powers), 3, 2, D, rot, dtype, seed=D)
    x = s["q"].double()
    x = torch.where(x < 0, -1.0, 1.0) * (1 + x.abs().frac() * 0.98) * torch.exp2(torch.tensor(powers, device="cuda").double())[:, None, None]
    x = x.to(dtype)
    assert torch.isfinite(x).all()
    want = expect(x, s["pos"], s["freq"], s["wq"], interleaved)
    assert want[0].abs().amax() < 16
    got = dsp.rope_store(x, None, None, s["pos"], s["freq"], q_weight=s["wq"], eps=EPS, interleaved=interleaved)["q"]
    near(got, *want, D, True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,rot", LAYOUTS)
def test_large_and_small_in_one_head(dtype, D, rot):
    """A few elements of 2^127, the rest 1 to 2^100: what is left of those is right too, down to
    the type's smallest normal numbers.  (Below, roundings are by 2^-134 in bf16, and by 2^-150 each in fp32.)"""
    s = case(6, 3, 2, D, rot, dtype, seed=D + 1)
    x = s["q"].double() * torch.exp2(torch.tensor([0, 20, 60, 80, 100, 110], device="cuda").double())[:, None, None]
    x[..., D // 2] = 2.0 ** 127
    x[:, 1, 0] = -2.0 ** 126
    x = x.to(dtype)
    want, size = expect(x, s["pos"], s["freq"], s["wq"], False)
    got = dsp.rope_store(x, None, None, s["pos"], s["freq"], q_weight=s["wq"], eps=EPS)["q"]
    near(got, want, size + 2.0 ** (-114 if dtype == torch.bfloat16 else -126), D, True)  # 16 u 2^-114 = 2^-134


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,rot", LAYOUTS)
def test_only_the_large_heads_of_the_normed_kind(dtype, D, rot):
    """Large heads beside others in one warp, a norm of the queries or of the keys alone, with the
    cache: the other heads and the values are as they are without the large ones, bit for bit."""
    s = case(7, 5, 3, D, rot, dtype, seed=D + 2)
    q, k, v = (s[n].clone() for n in "qkv")
    for x, h in ((q, 1), (q, 4), (k, 2), (v, 0)):
        x[:, h] = (x[:, h].double() * 2.0 ** 70).to(dtype)
    page, off = s["slot"].long() // s["page"], s["slot"].long() % s["page"]
    for weights in (dict(q_weight=s["wq"]), dict(k_weight=s["wk"]), dict(q_weight=s["wq"], k_weight=s["wk"])):
        got = {}
        for name, (a, b, c) in (("plain", (s["q"], s["k"], s["v"])), ("large", (q, k, v))):
            kc, vc = (t.clone() for t in s["caches"])
            o = dsp.rope_store(a, b, c, s["pos"], s["freq"], slot=s["slot"], k_cache=kc, v_cache=vc, eps=EPS, **weights)
            got[name] = (o["q"], kc[page, :, off], vc[page, :, off])
        for i, others in enumerate(([0, 2, 3], [0, 1], [1, 2])):
            assert torch.equal(got["large"][i][:, others], got["plain"][i][:, others])
        assert torch.equal(got["large"][2], v)
        near(got["large"][0], *expect(q, s["pos"], s["freq"], weights.get("q_weight"), False), D, True)
        near(got["large"][1], *expect(k, s["pos"], s["freq"], weights.get("k_weight"), False), D, True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [256, 128, 9])
def test_eps_counts_beside_large_squares(dtype, D):
    """eps of 9e29, above 2^-21 of a mean whose sum is just beyond fp32, and of 1e29 beside a
    mean of 1e30."""
    s = case(4, 2, 1, D, 0, dtype, seed=D + 3)
    for size in ((3.5e38 / D) ** 0.5, 1e15):
        x = (torch.where(s["q"] < 0, -1.0, 1.0) * size).to(dtype)
        for eps in (9e29, 1e29):
            got = dsp.rope_store(x, None, None, s["pos"], s["freq"], q_weight=s["wq"], eps=eps)["q"]
            near(got, *expect(x, s["pos"], s["freq"], s["wq"], False, eps), D, True)
