"""tree_attention4 against softmax in 64 bits over the values that the cache stands for.

Tolerances, from the inputs: a score is a sum of D products in fp32, off by at most
ds = D 2^-24 scale sum |q k|; a weight by a factor within exp(+-(ds + 1e-6)) (ex2, its
argument's rounding at |s| below 2^5); the output, a weighted mean, by 2 (ds + 1e-6)
max|v|, and, with a sum over n tokens in fp32 in tiles, by 2^-24 (sqrt(n) + 64) max|v|
more.  bf16 rounds each weight by at most 2^-8 of it, so a weighted mean by at most 2^-8
max|v|, and the result, 2^-8 |out|.  The log-sum-exp: ds + 1e-6 (1 + |lse|)."""
import numpy as np
import pytest
import torch

import cache4_plain as c4
import speculative_decoding_drafter_markov_gb300 as dsp
from speculative_decoding_drafter_markov_gb300 import _lib
from test_gpu_target import INF, err_word, expect, ints, make, shifted

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]


def hold(s):
    """The case with its caches in 4 bits (k4, v4) and their values (kc, vc, fp32)."""
    s = dict(s)
    for name in "kv":
        cache, values = c4.cache_of(s[name + "c"].double().cpu().numpy())
        s[name + "4"] = torch.from_numpy(cache).cuda()
        s[name + "c"] = torch.from_numpy(values).float().cuda()
    return s


def make4(*args, **kw):
    return hold(make(*args, **kw))


def call(s, **kw):
    err = err_word()
    out = dsp.tree_attention4(s["q"], s["k4"], s["v4"], s["table"], ints(s["lens"]), ints(s["start"]), mask=s["mask"],
                              scale=s["scale"], max_rows=max(s["rows"]), err=err, **kw)
    return out, err


def check(s, got, err, want=None):
    out, lse, ds, vmax = want or expect(s)
    assert int(err) == 0
    o, lg = got["out"].double(), got["lse"].double()
    n = max(a + b for a, b in zip(s["lens"], s["rows"]))
    fine = torch.isfinite(out)
    assert torch.equal(torch.isfinite(o), fine) and torch.equal(o.isnan(), out.isnan())
    tol = ((2 * (ds + 1e-6) + 2.0 ** -24 * (n ** 0.5 + 64)) * vmax)[:, :, None].expand_as(out)
    if s["q"].dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (vmax[:, :, None] + out.abs())
    assert ((o - out).abs()[fine] <= tol[fine]).all(), float(((o - out).abs() / tol.clamp(min=1e-30))[fine].max())
    ok = torch.isfinite(lse)
    assert torch.equal(lg[~ok & ~lse.isnan()], lse[~ok & ~lse.isnan()]) and torch.equal(lg.isnan(), lse.isnan())
    assert ((lg - lse).abs()[ok] <= (ds + 1e-6 * (1 + lse.abs()))[ok]).all()


LAYOUTS = [(1, 1, 64, 16), (8, 2, 128, 16), (32, 8, 128, 32), (7, 1, 128, 8), (6, 3, 80, 48), (12, 4, 96, 64), (4, 4, 64, 128),
           (8, 8, 128, 256), (2, 1, 16, 16), (3, 1, 48, 8), (5, 5, 80, 8), (4, 2, 256, 16), (16, 2, 208, 24), (2, 2, 112, 16), (64, 4, 128, 16),
           (34, 2, 32, 40), (2, 1, 128, 3), (256, 2, 64, 16)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,H,D,page", LAYOUTS)
def test_layouts(dtype, Hq, H, D, page):
    """Ragged chains: caches of none, one and many tokens, ends inside pages and tiles."""
    s = make4([0, 1, 127, 128, 129, 63, 700, 0], [1, 5, 1, 3, 9, 2, 17, 4], Hq, H, D, page, dtype, seed=D + page)
    check(s, *call(s))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,D", [(8, 128), (2, 64), (16, 96)])
def test_single_rows(dtype, Hq, D):
    """Plain decoding: one row of each request."""
    lens = [0, 1, 2, 126, 127, 128, 255, 256, 1000, 31]
    s = make4(lens, [1] * len(lens), Hq, 2, D, 16, dtype, seed=D)
    check(s, *call(s))


@pytest.mark.parametrize("Hq,H,D,page,rows", [(16, 1, 128, 16, 1), (9, 1, 64, 16, 1), (24, 2, 96, 16, 4), (6, 2, 128, 8, 5), (48, 2, 64, 32, 2), (20, 1, 80, 16, 2),
                                              (4, 1, 128, 16, 12), (15, 5, 48, 16, 3), (40, 1, 128, 64, 1), (2, 2, 32, 16, 48), (17, 1, 128, 16, 2)])
def test_few_lines(Hq, H, D, page, rows):
    """Units of 8 and of 16 lines: groups that fill them, that leave some over, that take several."""
    lens = [0, 40, 700, 64, 1500, 31, 33]
    for tree in (False, True):
        s = make4(lens, [rows, 1, max(1, rows - 1), rows, (rows + 1) // 2, rows, 1], Hq, H, D, page, torch.bfloat16, seed=Hq + D, tree=tree)
        check(s, *call(s))


def test_no_rows_at_all():
    s = make4([50, 0, 7], [1, 1, 1], 4, 2, 64, 16, torch.bfloat16)
    out = {"out": torch.full((3, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda"), "lse": torch.full((3, 4), 7.0, device="cuda")}
    for rows in (1, 40):
        err = err_word()
        dsp.tree_attention4(s["q"], s["k4"], s["v4"], s["table"], ints(s["lens"]), ints([0, 0, 0, 0]), max_rows=rows, out=out, err=err)
        assert int(err) == 0 and (out["out"] == 7).all() and (out["lse"] == 7).all()


@pytest.mark.parametrize("rows", [[2, 1, 1], [40, 2, 30]])
def test_two_at_once(rows):
    """Two calls on two streams, each with a workspace of its own, and again on one."""
    cases = [make4([2000, 40, 333], rows, 8, 2, 128, 16, torch.bfloat16, seed=i) for i in range(2)]
    want = [expect(s) for s in cases]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        got = [call(s, stream=side) for s, side in zip(cases, sides)]
        torch.cuda.synchronize()
        for s, (o, err), w in zip(cases, got, want):
            check(s, o, err, w)
    for s, w in zip(cases, want):
        check(s, *call(s), w)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,ctx,G", [(1, 0, 4), (64, 100, 1), (65, 127, 2), (128, 300, 4), (256, 1000, 3), (200, 5, 8)])
def test_trees(dtype, n, ctx, G):
    s = make4([ctx, 2 * ctx + 3, ctx], [n, 7, max(1, n // 2)], 2 * G, 2, 64, 16, dtype, seed=n, tree=True)
    check(s, *call(s))


@pytest.mark.parametrize("dtype", TYPES)
def test_long_chain(dtype):
    """A prompt in one call: more lines than a unit holds, every row a longer view."""
    s = make4([0, 300], [401, 3], 4, 2, 128, 16, dtype, seed=3)
    check(s, *call(s))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,ctx,rows", [(1, 20000, 1), (1, 20000, 40), (3, 9000, 3), (200, 50, 3)])
def test_split_and_packed(dtype, R, ctx, rows):
    """One cache over many CTAs, and many caches in one."""
    rng = np.random.default_rng(R)
    lens = [int(rng.integers(ctx // 2, ctx + 1)) for _ in range(R)]
    s = make4(lens, [int(rng.integers(1, rows + 1)) for _ in range(R)], 8, 4, 128, 32, dtype, seed=R)
    check(s, *call(s))


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("lens,rows", [([3000, 10, 700, 0, 129, 5000], [1, 40, 64, 3, 65, 17]), ([0, 0, 0], [33, 1, 64]),
                                       ([20000, 127], [64, 32]), ([60] * 40, [34, 2, 64, 30] * 10), ([900, 5, 64, 2000], [16, 3, 12, 1])])
def test_small_and_large_blocks(tree, lens, rows):
    s = make4(lens, rows, 8, 2, 128, 16, torch.bfloat16, seed=len(lens), tree=tree)
    check(s, *call(s))


@pytest.mark.parametrize("hint", [1, 5, 16, 17, 32, 33, 64, 300])
def test_hints(hint):
    """max_rows is a hint: any gives the same result but for roundings."""
    s = make4([300, 1000, 20], [33, 5, 70], 8, 2, 128, 16, torch.bfloat16, seed=4)
    err = err_word()
    got = dsp.tree_attention4(s["q"], s["k4"], s["v4"], s["table"], ints(s["lens"]), ints(s["start"]), scale=s["scale"], max_rows=hint, err=err)
    check(s, got, err)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("spread", [0.0, 30.0])
def test_flat_and_peaked(dtype, spread):
    s = make4([900, 40, 3000], [5, 2, 1], 8, 2, 64, 16, dtype, seed=1, spread=spread)
    check(s, *call(s))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [5, 40])
def test_scores_that_rise(dtype, rows):
    """Keys that grow along the text: the running maximum moves in every tile."""
    s = make([2500, 700], [rows, 2], 8, 2, 128, 16, dtype, seed=2)
    for r, (a, b) in enumerate(zip(s["lens"], s["rows"])):
        t = torch.arange(a + b, device="cuda")
        pg = s["table"][r].long()[t // 16]
        s["kc"][pg, :, t % 16] = (s["q"][0, ::4] * (t[:, None, None] / 150.0)).to(dtype)
    s = hold(s)
    check(s, *call(s))


@pytest.mark.parametrize("dtype", TYPES)
def test_sizes_of_scales(dtype):
    """Keys and values near both ends of the scales' range."""
    for k_size, v_size in ((1e-4, 1e5), (3e3, 2e-4)):
        s = make([300, 77], [3, 2], 4, 2, 64, 16, dtype, seed=6)
        s["kc"] *= k_size
        s["vc"] *= v_size
        s["scale"] = 0.125 / k_size
        s = hold(s)
        check(s, *call(s))


@pytest.mark.parametrize("dtype", TYPES)
def test_requests_without_rows(dtype):
    s = make4([50, 10, 0, 99], [0, 3, 0, 2], 4, 2, 64, 16, dtype)
    check(s, *call(s))


@pytest.mark.parametrize("dtype", TYPES)
def test_empty_rows(dtype):
    """A mask that leaves nothing: zeros and -inf, whatever stands in the cache."""
    for rows in ([6, 70, 5], [6, 9, 5]):
        s = make4([0, 0, 40], rows, 8, 2, 128, 16, dtype, tree=True)
        last = rows[0] + rows[1] - 1
        for i in (0, 3, last, last + 1):  # the last one of the cached request: the cache alone
            s["mask"][i] = 0
        want = expect(s)
        got, err = call(s)
        check(s, got, err, want)
        for i in (0, 3, last):
            assert not got["out"][i].any() and (got["lse"][i] == -INF).all()
        s["v4"].fill_(255)  # NaN throughout
        got, _ = call(s)
        for i in (0, 3, last):
            assert not got["out"][i].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ctx,n,tree", [(37, 20, True), (120, 9, False), (0, 130, True), (128, 64, True), (500, 3, False), (300, 12, True)])
def test_what_is_not_seen_has_no_influence(dtype, ctx, n, tree):
    """Stale slots and rows that others do not see hold NaN."""
    nan = float("nan")
    s = make([ctx, 11], [n, 2], 8, 2, 128, 16, dtype, seed=n, tree=tree, extra=3)
    bad = torch.ones(s["kc"].shape[0], s["page"], dtype=torch.bool, device="cuda")
    for r, (a, b) in enumerate(zip(s["lens"], s["rows"])):
        for t in range(a + b):
            bad[int(s["table"][r, t // s["page"]]), t % s["page"]] = False
    for c in ("kc", "vc"):
        s[c][bad[:, None, :].expand(s[c].shape[:3])] = nan
    h = hold(s)
    check(h, *call(h))
    # a row of the cycle itself: those that see it, and they alone, are touched, in the 16 columns of its scale
    t = ctx + n - 2 if n > 2 else ctx + 1
    pg, off = int(s["table"][0, t // s["page"]]), t % s["page"]
    s["vc"][pg, :, off, [3, 40]] = nan
    h = hold(s)
    want = expect(h)
    assert want[0].isnan().any() and not want[0][..., 48:].isnan().any()
    check(h, *call(h), want)
    s["kc"][pg, :, off] = nan
    h = hold(s)
    want = expect(h)
    got, err = call(h)
    seen = want[1].isnan()
    assert seen.any() and not seen.all()
    assert got["lse"][seen].isnan().all() and torch.equal(got["lse"].isnan(), seen)
    assert got["out"][seen].isnan().all()
    check(dict(h, q=h["q"]), {k: torch.where(seen if v.dim() == 2 else seen[..., None], want[i].to(v.dtype), v) for i, (k, v) in
                              enumerate(got.items())}, err, want)


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes, its last pages in use."""
    H, page, D = 8, 64, 128
    n_pages = (1 << 32) // (H * page * D * 9 // 16) + 40
    for dtype in TYPES:
        small = make4([700, 300], [3, 9], 16, H, D, page, dtype, seed=5, extra=0)
        n = small["k4"].shape[0]
        big = {}
        for c in ("k4", "v4"):
            big[c] = dsp.cache4(n_pages, H, page, D)
            big[c][-n:] = small[c]
        want = expect(small)
        s = dict(small, table=torch.where(small["table"] >= 0, small["table"] + n_pages - n, -1).int(), **big)
        check(s, *call(s), want)


@pytest.mark.parametrize("rows", [[5, 2, 1], [40, 2, 1]])
def test_on_another_stream_and_in_a_graph(rows):
    s = make4([900, 40, 3], rows, 8, 2, 128, 16, torch.bfloat16, seed=1)
    want = expect(s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, err = call(s, stream=side)
    side.synchronize()
    check(s, got, err, want)
    lens, start, err = ints(s["lens"]), ints(s["start"]), err_word()
    args = (s["q"], s["k4"], s["v4"], s["table"], lens, start)
    ws = torch.empty(dsp.tree_attention4_workspace_size(*args, max_rows=max(rows)), dtype=torch.uint8, device="cuda")
    out = {"out": torch.zeros(s["q"].shape, dtype=s["q"].dtype, device="cuda"), "lse": torch.zeros(s["q"].shape[:2], device="cuda")}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsp.tree_attention4(*args, max_rows=max(rows), out=out, ws=ws, err=err)
    ws.fill_(0xFF)  # nothing is kept in the workspace from call to call
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    check(s, out, err, want)
    # shorter caches in the same graph: lengths are read on the GPU
    s2 = dict(s, lens=[100, 0, 2])
    lens.copy_(ints(s2["lens"]))
    graph.replay()
    torch.cuda.synchronize()
    check(s2, out, err)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("most", [4, 40])
def test_device_side_errors(dtype, most):
    """Sizes and pages out of range are reported; the other requests' rows are right."""
    s = make4([60, 30, 90], [3, 2, most], 4, 2, 64, 16, dtype, seed=2)
    want = expect(s)
    for change in ("long", "negative", "page", "minus"):
        lens, table = list(s["lens"]), s["table"].clone()
        if change == "long":
            lens[1] = 10 ** 9
        elif change == "negative":
            lens[1] = -5
        else:
            table[1, 0] = 1 << 30 if change == "page" else -1
        err = err_word()
        got = dsp.tree_attention4(s["q"], s["k4"], s["v4"], table, ints(lens), ints(s["start"]), scale=s["scale"], max_rows=most, err=err)
        assert int(err) == _lib.ERR_RANGE
        keep = [0, 1, 2] + list(range(5, 5 + most))
        check(dict(s, q=s["q"][keep]), {k: v[keep] for k, v in got.items()}, err_word(), tuple(w[keep] for w in want))


def test_rows_beyond_the_batch_stay():
    s = make4([60, 30], [3, 2], 4, 2, 64, 16, torch.bfloat16, seed=2)
    q = torch.cat([s["q"], s["q"]])
    out = {"out": torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda"), "lse": torch.full(q.shape[:2], 7.0, device="cuda")}
    dsp.tree_attention4(q, s["k4"], s["v4"], s["table"], ints(s["lens"]), ints(s["start"]), scale=s["scale"], out=out)
    assert (out["out"][5:] == 7).all() and (out["lse"][5:] == 7).all()
    check(s, {k: v[:5] for k, v in out.items()}, err_word())


PAGE = 45691136  # 47 of them are the 2^31 - 256 tokens that a table may name


def one_long_page():
    """Caches of one page, keys and values of 0: codes of 8."""
    pair = [dsp.cache4(1, 1, PAGE, 16) for _ in range(2)]
    for cache in pair:
        cache[:, :, :PAGE * 8] = 0x88
    return pair


@pytest.mark.parametrize("R,hint", [(43, 1), (5, 300)])
def test_tokens_to_the_end_of_32_bits(R, hint):
    """Caches whose tokens are 47 times the same page, the last one a table may name.  Keys of
    zero, values of 0 but for a few that hold 63/64 for 1 (7 times the scale 9/64) in each column: sums of
    whole numbers of 63 2^-6 (of their eighths, times a weight of 2^7: of 1/4) below 2^24 of those, and means.
    Partials are joined in fp32, eight at most at a time: 8 2^-24."""
    kc, vc = one_long_page()
    rng = np.random.default_rng(1)
    count = [1, 100, 5000, 70000, 200000, 17, 2, 0]
    rows = {}
    for d, n in enumerate(count):
        at = np.unique(np.concatenate([[0] * (n > 0), rng.integers(1, PAGE - 1, 2 * n)])).astype(np.int64)[:n]
        at[1:][-1:] = PAGE - 1
        rows[d] = at
    slots = np.unique(np.concatenate(list(rows.values())))
    v = np.zeros((len(slots), 1, 16), np.float32)
    for d, at in rows.items():
        v[np.searchsorted(slots, at), 0, d] = 1
    v = torch.from_numpy(v).cuda()
    dsp.cache_store4(torch.zeros_like(v), v, ints(slots), kc, vc)
    tokens, err = PAGE * 47, err_word()
    assert tokens == 0x7fffff00
    q = torch.ones((R, 1, 16), dtype=torch.bfloat16, device="cuda")
    got = dsp.tree_attention4(q, kc, vc, torch.zeros((R, 47), dtype=torch.int32, device="cuda"), ints([tokens - 1] * R), ints(list(range(R + 1))),
                              max_rows=hint, err=err)
    assert int(err) == 0
    want = torch.tensor(count + [0] * 8, dtype=torch.float64, device="cuda") * (63 / 64) / PAGE
    assert ((got["out"].double() - want).abs() <= (2.0 ** -8 + 8 * 2.0 ** -24) * want).all()
    lse = np.log(float(tokens))
    assert ((got["lse"].double() - lse).abs() <= 1e-6 * (1 + lse)).all()


def test_calls_of_hours_are_refused():
    """8192 caches of 2^31 - 256 tokens: reported, and no row is written."""
    R, (kc, vc), err = 8192, one_long_page(), err_word()
    out = {"out": torch.full((R, 1, 16), 7.0, dtype=torch.bfloat16, device="cuda"), "lse": torch.full((R, 1), 7.0, device="cuda")}
    dsp.tree_attention4(torch.ones((R, 1, 16), dtype=torch.bfloat16, device="cuda"), kc, vc, torch.zeros((R, 47), dtype=torch.int32, device="cuda"),
                        ints([PAGE * 47 - 1] * R), ints(list(range(R + 1))), out=out, err=err)
    assert int(err) == _lib.ERR_UNSUPPORTED and (out["out"] == 7).all() and (out["lse"] == 7).all()


def test_same_bits_again():
    for rows in ([5, 2, 1], [33, 2, 1]):
        s = make4([9000, 40, 333], rows, 8, 2, 128, 16, torch.bfloat16, seed=1)
        a, _ = call(s)
        for _ in range(3):
            b, _ = call(s)
            assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [0.0, -0.25, 0.5])
@pytest.mark.parametrize("most", [40, 5])
def test_scales(dtype, scale, most):
    s = make4([300, 0, 77], [3, 2, most], 8, 2, 64, 16, dtype, seed=3, tree=True)
    s["scale"] = scale
    check(s, *call(s))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("what", ["q", "q_row", "q_head", "out", "heads", "one"])
def test_addresses(dtype, what):
    s = make4([300, 0, 77], [3, 2, 40], 8, 2, 64, 16, dtype, seed=4)
    s["q"] = s["q"].contiguous()
    N, Hq, D = s["q"].shape
    kw = {}
    if what == "q":
        s["q"] = shifted(s["q"])
    elif what == "out":
        kw["out"] = {"out": shifted(s["q"]), "lse": torch.empty((N, Hq), device="cuda")}
    elif what == "heads":
        s["q"] = s["q"].transpose(0, 1).contiguous().transpose(0, 1)
    elif what == "one":
        s["q"] = s["q"][:1].expand(N, -1, -1)
    else:
        wide = torch.zeros((N, Hq * D + 1) if what == "q_row" else (N, Hq, D + 3), dtype=dtype, device="cuda")
        view = wide[:, :Hq * D].view(N, Hq, D) if what == "q_row" else wide[:, :, :D]
        view.copy_(s["q"])
        s["q"] = view
    check(s, *call(s, **kw))


def test_refusals():
    s = make4([60, 30], [3, 2], 4, 2, 64, 16, torch.bfloat16)
    ok = (s["q"], s["k4"], s["v4"], s["table"], ints(s["lens"]), ints(s["start"]))
    for bad in [(s["q"].transpose(1, 2), *ok[1:]), (ok[0], s["k4"].cpu(), *ok[2:]), (*ok[:5], ok[5][:-1]), (*ok[:2], s["v4"][1:], *ok[3:]),
                (s["q"][..., :40], *ok[1:]), (ok[0], s["k4"][:, :, :-16].contiguous(), *ok[2:]), (*ok[:1], s["kc"], *ok[2:])]:
        with pytest.raises(ValueError):
            dsp.tree_attention4(*bad)
    for bad in [(s["q"].half(), *ok[1:]), (ok[0], s["k4"].view(torch.int8), *ok[2:]), (*ok[:4], ok[4].long(), ok[5])]:
        with pytest.raises(TypeError):
            dsp.tree_attention4(*bad)
    with pytest.raises(ValueError):
        dsp.tree_attention4(*ok, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(dsp.DSparkError):
        dsp.tree_attention4(s["q"][:, :3], *ok[1:])
    ws = torch.empty(dsp.tree_attention4_workspace_size(*ok) + 64, dtype=torch.uint8, device="cuda")
    with pytest.raises(dsp.DSparkError, match="workspace"):
        dsp.tree_attention4(*ok, ws=ws[8:])
    err = err_word()
    check(s, dsp.tree_attention4(*ok, scale=s["scale"], ws=ws[16:], err=err), err)
    assert dsp.tree_attention4(s["q"][:0], s["k4"], s["v4"], s["table"], ok[4], ints([0, 0, 0]))["out"].shape == (0, 4, 64)
