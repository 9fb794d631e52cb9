"""The attention's weights and values, closer than by the largest value.

Tolerances, from the arithmetic.  With A = sum_t softmax(s)_t |v_t| per row, head
and column, n tokens and u = 2^-24:
* a score is off by at most ds = D u scale sum|q k| (see `expect`), a weight by
  exp(+-(ds + 1e-6)), numerator and sum together 2 (ds + 1e-6) A;
* bf16: the weight that multiplies the values is rounded, by at most 2^-8 of it
  (eight significant bits): 2^-8 A at worst.  The roundings of n weights are of
  either sign and independent, so they add up on the 2-norm B = (sum_t
  (softmax(s)_t v_t)^2)^(1/2): beyond 6 2^-8 B with a probability below
  2 exp(-18) (Hoeffding), a bound that shrinks with n where the first does not;
* products are exact, and a sum in the tensor cores loses at most 2 u of its size
  at each of n / 16 steps, one on the CUDA cores at most u at each of n: n u A;
  joins and the final product: 32 u A;
* bf16: the result is rounded once, by at most half of its last place: 2^-8 |out|.

With keys of zero and values of +-1 every weight is 1, every sum a whole number
below 2^24, so nothing is rounded before the division: 4 u |out| and the bf16.
"""
import os
import subprocess
import sys
import tempfile

import numpy as np
import pytest
import torch

import speculative_decoding_drafter_markov_gb300 as dsp
from test_gpu_target import call, expect, make

pytestmark = pytest.mark.gpu


def sizes(s):
    """(A, B): sum and 2-norm of the weighted values, in 64 bits."""
    A = expect(dict(s, vc=s["vc"].abs()))[0]
    # twice the scores: weights in proportion to the squares, of which the sums are known
    _, lse, _, _ = expect(s)
    square, lse2, _, _ = expect(dict(s, vc=s["vc"].double().square(), scale=2 * s["scale"]))
    return A, (square * torch.exp(lse2 - 2 * lse)[:, :, None]).sqrt()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128, 96])
@pytest.mark.parametrize("lens,rows,tree", [([0, 20, 127, 300], [3, 1, 9, 17], False), ([130, 40], [64, 33], True),
                                            ([1500], [5], False), ([60] * 12, [4] * 12, False)])
def test_weights_keep_their_precision(dtype, D, lens, rows, tree):
    """Many weights of one size, whose errors show in the small outputs."""
    s = make(lens, rows, 8, 2, D, 16, dtype, seed=D + len(lens), tree=tree, spread=0.125)
    out, _, ds, _ = expect(s)
    A, B = sizes(s)
    n = max(a + b for a, b in zip(lens, rows))
    got, err = call(s)
    assert int(err) == 0
    tol = (2 * (ds + 1e-6) + (n + 32) * 2.0 ** -24)[:, :, None] * A
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (torch.minimum(6 * B, A) + out.abs())
    off = (got["out"].double() - out).abs()
    assert (off <= tol).all(), float((off / tol).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,D", [(4, 128), (2, 64)])
@pytest.mark.parametrize("lens,rows,tree", [([20000], [3], False), ([9000, 5000], [40, 2], True), ([700, 3000, 0], [64, 1, 200], True),
                                            ([3000], [300], False)])
def test_every_tile_of_values_counts(dtype, G, D, lens, rows, tree):
    """Keys of zero, values of +-1: the output is a mean, and each tile of it shows."""
    s = make(lens, rows, 2 * G, 2, D, 16, dtype, seed=len(lens) + D, tree=tree)
    s["kc"].zero_()
    s["vc"].copy_(torch.where(s["vc"] < 0, -1.0, 1.0))
    N = s["q"].shape[0]
    # means on the CPU from the tables and masks, in 64 bits
    v = s["vc"].cpu().double().numpy()
    table, page, start = s["table"].cpu().numpy(), s["page"], s["start"]
    want, wrong = (np.zeros((N, 2 * G, D)) for _ in range(2))
    for r, (n_ctx, n) in enumerate(zip(lens, rows)):
        t = np.arange(n_ctx + n)
        vals = v[table[r, t // page], :, t % page]  # [tokens, H, D]
        cache = vals[:n_ctx].sum(0)
        # the same with the values of a tile taken from another one: what the test has to see
        tile = cache - vals[:128].sum(0) + vals[n_ctx - 128:n_ctx].sum(0) if n_ctx >= 256 else cache
        for j in range(n):
            i = start[r] + j
            if s["mask"] is None:
                seen = np.arange(j + 1)
            else:
                w = [int(x) for x in s["mask"][i]]
                seen = np.array([u for u in range(n) if (w[u // 64] >> (u % 64)) & 1])
            own = vals[n_ctx + seen].sum(0)
            for out, part in ((want, cache), (wrong, tile)):
                out[i] = ((part + own) / (n_ctx + len(seen))).repeat(G, 0)
    got, err = call(s)
    assert int(err) == 0
    g = got["out"].double().cpu().numpy()
    tol = 4 * 2.0 ** -24 * np.abs(want) + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0)
    assert (np.abs(g - want) <= tol).all()
    for r, n_ctx in enumerate(lens):
        if n_ctx >= 256:
            rows_r = slice(start[r], start[r + 1])
            assert (np.abs(wrong - want)[rows_r] > 2 * tol[rows_r]).mean() > 0.5


def test_tokens_to_the_end_of_32_bits():
    """43 caches whose 2^31 - 256 tokens are 47 times the same page: the last token that
    a table may name, and a line of more than 2^31 places.  Keys of zero, values of 0
    but for a few of 1 in each column: sums of whole numbers below 2^24, and means.
    Partials of the sums and weights are joined in fp32, four at most: 8 2^-24."""
    R, page, pages, D = 43, 45691136, 47, 8
    kc, vc = (torch.zeros((1, 1, page, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rng = np.random.default_rng(1)
    count = [1, 100, 5000, 70000, 300000, 17, 2, 0]
    for d, n in enumerate(count):  # the first token of the page, some others and the last
        at = np.unique(np.concatenate([[0] * (n > 0), rng.integers(1, page - 1, 2 * n)])).astype(np.int64)[:n]
        at[1:][-1:] = page - 1
        vc[0, 0, torch.from_numpy(at).cuda(), d] = 1
    tokens = page * pages
    assert tokens == 0x7fffff00
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    err = ints([0])
    q = torch.ones((R, 1, D), dtype=torch.bfloat16, device="cuda")
    got = dsp.tree_attention(q, kc, vc, torch.zeros((R, pages), dtype=torch.int32, device="cuda"), ints([tokens - 1] * R),
                             ints(list(range(R + 1))), err=err)
    assert int(err) == 0
    want = torch.tensor(count, dtype=torch.float64, device="cuda") / page
    assert ((got["out"].double() - want).abs() <= (2.0 ** -8 + 8 * 2.0 ** -24) * want).all()
    lse = np.log(float(tokens))
    assert ((got["lse"].double() - lse).abs() <= 1e-6 * (1 + lse)).all()


def test_the_drafts_switch_is_the_drafts():
    """DSPARK_DRAFT_KERNEL chooses the draft's kernel; the attention's results are the same bits."""
    code = """
import sys, torch
from test_gpu_target import call, make
s = make([700, 40, 3], [5, 2, 1], 8, 2, 128, 16, torch.bfloat16, seed=1)
out, err = call(s)
torch.save((out["out"].cpu(), out["lse"].cpu()), sys.argv[1])
"""
    here = os.path.dirname(os.path.abspath(__file__))
    path = os.pathsep.join([here, os.path.dirname(here)])
    got = []
    for value in (None, "simt"):
        env = {k: v for k, v in os.environ.items() if k != "DSPARK_DRAFT_KERNEL"}
        if value:
            env["DSPARK_DRAFT_KERNEL"] = value
        with tempfile.NamedTemporaryFile(suffix=".pt") as f:
            subprocess.run([sys.executable, "-c", code, f.name], env=dict(env, PYTHONPATH=path), check=True)
            got.append(torch.load(f.name))
    assert all(torch.equal(a, b) for a, b in zip(*got))
