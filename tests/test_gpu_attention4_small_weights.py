"""tree_attention4 where nearly all weights of a row are small beside its largest.

Weights are rounded to fp16 for the product with the values, the largest of a row so far at 2^7 or
above when the reference is set: by 2^-11 of a weight that is 2^-21 of the row's largest or more
(fp16's normal numbers), by 2^-25 / 2^7 = 2^-32 of the largest below that.  Weights of one size are all
rounded in one direction: n of them lose 2^-32 n of the largest at worst, times their value."""
import math

import pytest
import torch

import speculative_decoding_drafter_markov_gb300 as dsp
from test_gpu_target import err_word, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,n", [(256, 4096), (3, 1 << 18)])
@pytest.mark.parametrize("hint", [2, 12, 13, 40])
def test_a_flat_tail_behind_one_large_weight(R, n, hint):
    """One token whose value is zero and n - 1 behind it whose weights are 2^-x of its: fp16's normal
    numbers, then its subnormal ones, then none of them.  With 256 requests of 8 heads a share holds
    whole caches.  Scores are products of powers of two and the scale alone is rounded: x is off by
    x 2^-23, a weight by x 2^-23 of it, ex2 by 2^-22 more, and all of a tail in one direction."""
    H, G, D, page, up = 8, 4, 64, 256, 4.0
    k, v = (torch.zeros((2 * page, H, D), device="cuda") for _ in range(2))
    k[0, :, 0] = 7.0     # scale 1, code 7
    v[page:] = 63 / 64
    v[1:page] = 63 / 64  # page 0: the first one of every cache; page 1: all others
    kc, vc = (dsp.cache4(2, H, page, D) for _ in range(2))
    held = dsp.cache_store4(k, v, torch.arange(2 * page, device="cuda", dtype=torch.int32), kc, vc, values=True)
    assert torch.equal(held["k"], k) and torch.equal(held["v"], v)
    table = torch.ones((R, n // page), dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    q = torch.zeros((R, H * G, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = up
    for x in (0.0, 10.25, 18.4, 22.6, 24.3, 27.8, 31.3, 40.0):
        scale, err = x * math.log(2) / (7 * up), err_word()
        got = dsp.tree_attention4(q, kc, vc, table, ints([n - 1] * R), ints(list(range(R + 1))), scale=scale, max_rows=hint, err=err)
        assert int(err) == 0
        tail, u = (n - 1) * 2.0 ** -x, 2.0 ** -24
        want = tail / (1 + tail) * 63 / 64
        tol = want * (2 * (2 * x * u + 4 * u) + (n + 32) * u + 2.0 ** -11 + 2.0 ** -8) + 2.0 ** -32 * n / (1 + tail)
        assert float((got["out"].double() - want).abs().max()) <= tol, x
        lse = x * math.log(2) + math.log1p(tail)
        assert float((got["lse"].double() - lse).abs().max()) <= 1e-6 * (2 + x + lse), x
