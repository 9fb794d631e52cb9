"""tree_attention4's weights and values, closer than by the largest value.

Tolerances, from the arithmetic.  With p_t = softmax(s)_t per row and head, A = sum_t p_t |v_t|
per column, n tokens and u = 2^-24:
* keys are exact in bf16, values in fp16; a score is off by at most ds = D u scale sum|q k|, a weight
  by exp(+-(ds + 1e-6)) (ex2, its argument's rounding at |s| below 2^5), numerator and sum
  together 2 (ds + 1e-6) A;
* the weight that multiplies the values is rounded to fp16, with the largest one of its row so far
  at 2^7 or above when the reference is set, and none above 2^15: by at most 2^-11 of a weight
  that is 2^-21 of the row's largest or more (fp16's normal numbers), by 2^-25 / 2^7 = 2^-32 of the
  largest below.  2^-11 A at worst; roundings of n weights are of either sign and independent, so they
  add up on B = (sum_t (p_t v_t)^2)^(1/2): beyond 6 2^-11 B with a probability below 2 exp(-18)
  (Hoeffding).  And 2^-32 max_t p_t sum_t |v_t| =: F, whatever the roundings' signs;
* products are exact, and a sum in the tensor cores loses at most 2 u of its size at each of
  n / 16 steps, a rescaling u of it: n u A; joins and the final product: 32 u A;
* the result is rounded once to bf16, by at most half of its last place: 2^-8 |out|.

With keys of zero and values of +-63/64 (7 times the scale 9/64) every weight is a power of two and
every sum a whole number of 63 2^-k below 2^24 of those: nothing is rounded before the division: 4 u
|out| and the bf16."""
import numpy as np
import pytest
import torch

from test_gpu_attention4 import call, hold
from test_gpu_target import make

pytestmark = pytest.mark.gpu


def plain(s, rounded=None):
    """(out, ds, A, B, F) per row, head and column in 64 bits; `rounded`: what the second product takes
    for the weights (relative to the row's largest), the sum being that of the weights themselves."""
    q = s["q"].double()
    N, Hq, D = q.shape
    H = s["kc"].shape[1]
    out, A, B, F = (torch.zeros((N, Hq, D), dtype=torch.float64, device="cuda") for _ in range(4))
    ds = torch.zeros((N, Hq, 1), dtype=torch.float64, device="cuda")
    for r, (n_ctx, n) in enumerate(zip(s["lens"], s["rows"])):
        t = torch.arange(n_ctx + n, device="cuda")
        k, v = (s[c][s["table"][r].long()[t // s["page"]], :, t % s["page"]].double().transpose(0, 1).repeat_interleave(Hq // H, 0)
                for c in ("kc", "vc"))
        for j in range(n):
            i = s["start"][r] + j
            see = torch.ones(n_ctx + n, dtype=torch.bool)
            words = None if s["mask"] is None else [int(w) for w in s["mask"][i]]
            for u in range(n):
                see[n_ctx + u] = u <= j if words is None else (words[u // 64] >> (u % 64)) & 1
            see = see.cuda()
            kk, vv = k[:, see], v[:, see]
            x = (kk @ q[i][:, :, None]).squeeze(-1) * s["scale"]
            w = torch.exp(x - x.amax(1, keepdim=True))
            total = w.sum(1, keepdim=True)
            out[i] = (((rounded(w) if rounded else w) / total)[:, None] @ vv).squeeze(1)
            p = (w / total)[:, None]
            A[i], B[i] = (p @ vv.abs()).squeeze(1), (p.square() @ vv.square()).squeeze(1).sqrt()
            F[i] = 2.0 ** -32 / total * vv.abs().sum(1)
            ds[i] = ((kk.abs() @ q[i].abs()[:, :, None]).amax(1) * abs(s["scale"])) * D * 2.0 ** -24
    return out, ds, A, B, F


def tolerance(s, out, ds, A, B, F):
    n = max(a + b for a, b in zip(s["lens"], s["rows"]))
    return (2 * (ds + 1e-6) + (n + 32) * 2.0 ** -24) * A + 2.0 ** -11 * torch.minimum(6 * B, A) + F + 2.0 ** -8 * out.abs()


# lines of 4 heads: up to 8, up to 48 (the warps' kernel); one operand and two of the other one
FEW, SOME = ([60, 200, 0] * 12, [2, 1, 2] * 12, False), ([0, 20, 127, 300], [3, 1, 9, 12], False)
ONE, TWO = ([0, 20, 200, 300], [3, 1, 9, 17], False), ([130, 40], [64, 33], True)


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("lens,rows,tree", [FEW, SOME, ([60] * 12, [4] * 12, True), ONE, TWO, ([300, 3], [40, 2], False)])
def test_weights_keep_their_precision(D, lens, rows, tree):
    """Many weights, whose errors show in the small outputs.  Weights in bf16 would not pass."""
    s = hold(make(lens, rows, 8, 2, D, 16, torch.bfloat16, seed=D + len(lens), tree=tree))
    want = plain(s)
    tol = tolerance(s, *want)
    got, err = call(s)
    assert int(err) == 0
    off = (got["out"].double() - want[0]).abs()
    assert (off <= tol).all(), float((off / tol).max())
    coarse = plain(s, lambda w: w.to(torch.bfloat16).double())[0].to(torch.bfloat16)
    assert ((coarse.double() - want[0]).abs() > tol).any()


@pytest.mark.parametrize("G,D", [(4, 128), (2, 64), (4, 96), (3, 80)])
@pytest.mark.parametrize("lens,rows,tree", [([20000], [2], False), ([9000, 5000], [12, 5], True), ([3000, 700] * 20, [1, 3] * 20, False),
                                            ([20000], [17], False), ([9000, 5000], [40, 2], True), ([700, 3000, 0], [64, 1, 200], True),
                                            ([3000], [300], False)])
def test_every_step_of_values_counts(G, D, lens, rows, tree):
    """The output is a mean of the values: each 32 tokens of it show."""
    s = make(lens, rows, 2 * G, 2, D, 16, torch.bfloat16, seed=len(lens) + D, tree=tree)
    s["kc"].zero_()
    s["vc"].copy_(torch.where(s["vc"] < 0, -1.0, 1.0))
    s = hold(s)
    v = s["vc"].cpu().double().numpy()
    assert (np.abs(v) == 63 / 64).all() and not s["kc"].any()
    table, page, start = s["table"].cpu().numpy(), s["page"], s["start"]
    want, wrong = (np.zeros((sum(rows), 2 * G, D)) for _ in range(2))
    for r, (n_ctx, n) in enumerate(zip(lens, rows)):
        t = np.arange(n_ctx + n)
        vals = v[table[r, t // page], :, t % page]  # [tokens, H, D]
        cache = vals[:n_ctx].sum(0)
        # the same with the values of one step taken from another: what the test has to see
        step = cache - vals[:32].sum(0) + vals[n_ctx - 32:n_ctx].sum(0) if n_ctx >= 64 else cache
        for j in range(n):
            i = start[r] + j
            words = None if s["mask"] is None else [int(x) for x in s["mask"][i]]
            seen = np.array([u for u in range(n) if (u <= j if words is None else (words[u // 64] >> (u % 64)) & 1)])
            own = vals[n_ctx + seen].sum(0)
            for out, part in ((want, cache), (wrong, step)):
                out[i] = ((part + own) / (n_ctx + len(seen))).repeat(G, 0)
    got, err = call(s)
    assert int(err) == 0
    tol = (4 * 2.0 ** -24 + 2.0 ** -8) * np.abs(want)
    assert (np.abs(got["out"].double().cpu().numpy() - want) <= tol).all()
    for r, n_ctx in enumerate(lens):
        if n_ctx >= 64:
            rows_r = slice(start[r], start[r + 1])
            assert (np.abs(wrong - want)[rows_r] > 2 * tol[rows_r]).mean() > 0.5
