"""GPU parity of the target-pass operators with plain implementations.

* page_map: against a simulator that moves the pages one by one; integers,
  compared exactly, over chained cycles, failures and repeated calls.
* cache_store: bits, from strided views, with skipped and bad slots.
* tree_attention: against softmax in 64 bits, at lengths, masks and layouts
  where it can go wrong.
* logit_rules: against the formula in 64 bits.

Tolerances of the attention, from the inputs: a score is a sum of D products in
fp32, off by at most ds = D 2^-24 scale sum|q k|; a weight by a factor within
exp(+-(ds + 1e-6)) (ex2, its argument's rounding at |s| below 2^5); the output,
a weighted mean, by 2 (ds + 1e-6) max|v|, and, with a sum over n tokens in fp32
in tiles, by 2^-24 (sqrt(n) + 64) max|v| more.  bf16 rounds the weights (2^-9 max|v|) and the
result (2^-9 |out|).  The log-sum-exp: ds + 1e-6 (1 + |lse|).
Of the rules: at most six fp32 roundings of terms no larger than the sum of
the terms' sizes, and one rounding to bf16.
"""
import numpy as np
import pytest
import torch

import speculative_decoding_drafter_markov_gb300 as dsp
from speculative_decoding_drafter_markov_gb300 import _lib

pytestmark = pytest.mark.gpu
INF = float("inf")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ page map
def tree_of(n, rng, back=8):
    return [-1 if j == 0 or rng.random() < 0.05 else int(rng.integers(max(0, j - back), j)) for j in range(n)]


def ancestors(parents):
    out = []
    for j, p in enumerate(parents):
        out.append((out[p] if p >= 0 else 0) | (1 << j))
    return out


def words_of(bits, W):
    return np.array([[(b >> (64 * w)) & 0xFFFFFFFFFFFFFFFF for w in range(W)] for b in bits], np.uint64).view(np.int64).reshape(-1, W)


class Sim:
    """The map by its definition, one page after the other."""

    def __init__(self, lens, rows, table, held, free, n_free, page, N, parents=None, W=0):
        need = [-(-(a + b) // page) for a, b in zip(lens, rows)]
        self.table, self.free, n = table.copy(), free.copy(), n_free
        back = [self.table[r, i] for r in range(len(rows)) for i in range(need[r], held[r])]
        for k, pg in enumerate(reversed(back)):
            self.free[n + k] = pg
        n += len(back)
        for r in range(len(rows)):
            for i in range(held[r], need[r]):
                n -= 1
                self.table[r, i] = self.free[n]
        self.held, self.n_free = need, n
        self.row_start = np.concatenate([[0], np.cumsum(rows)])
        self.slot, self.pos = np.full(N, -1), np.zeros(N, int)
        self.mask = np.zeros((N, W), np.int64)
        at = 0
        for r, n_rows in enumerate(rows):
            bits = ancestors(parents[at:at + n_rows]) if parents is not None else None
            for j in range(n_rows):
                t = lens[r] + j
                self.slot[at + j] = self.table[r, t // page] * page + t % page
                self.pos[at + j] = t if bits is None else lens[r] + bin(bits[j]).count("1") - 1
            if bits:
                self.mask[at:at + n_rows] = words_of(bits, W)
            at += n_rows


def check_map(out, table, free, sim):
    for k in ("held", "row_start", "slot", "pos"):
        assert np.array_equal(out[k].cpu().numpy(), getattr(sim, k)), k
    assert int(out["n_free"]) == sim.n_free
    assert np.array_equal(table.cpu().numpy(), sim.table)
    assert np.array_equal(free.cpu().numpy()[:sim.n_free], sim.free[:sim.n_free])
    if "mask" in out:
        assert np.array_equal(out["mask"].cpu().numpy(), sim.mask)


@pytest.mark.parametrize("R,page,most,tree", [(1, 16, 1, False), (5, 1, 3, True), (37, 16, 17, True), (513, 8, 5, False),
                                              (3000, 32, 2, True), (8192, 16, 1, False), (6, 24, 256, True)])
def test_map_cycles(R, page, most, tree):
    """Chained cycles: grow, accept a part, finish some requests, start others."""
    rng = np.random.default_rng(R + page)
    lens = rng.integers(0, 4 * page, R).astype(int).tolist()
    width = 4 + (4 * page + 6 * most) // page + most
    n_pages = R * (width - 1) + 3
    table, free = np.full((R, width), -1, np.int32), np.arange(n_pages, dtype=np.int32)
    rng.shuffle(free)
    held, n_free = [0] * R, n_pages
    t_d, f_d, h_d, n_d = torch.from_numpy(table).cuda(), torch.from_numpy(free).cuda(), ints(held), ints([n_pages])
    W = (most + 63) // 64
    err = err_word()
    for cycle in range(6):
        rows = rng.integers(0, most + 1, R).tolist()
        for r in rng.integers(0, R, max(1, R // 10)):  # finished
            lens[r] = rows[r] = 0
        N = sum(rows) + int(rng.integers(0, 5))
        parents = [p for n in rows for p in tree_of(n, rng)] if tree else None
        sim = Sim(lens, rows, table, held, free, n_free, page, N, parents, W)
        args = dict(page=page, N=N, parents=ints(parents) if tree else None, max_rows=most, err=err)
        out = dsp.page_map(ints(lens), ints(rows), t_d, h_d, f_d, n_d, **args)
        check_map(out, t_d, f_d, sim)
        again = dsp.page_map(ints(lens), ints(rows), t_d, h_d, f_d, n_d, **args)  # a call may be repeated
        check_map(again, t_d, f_d, sim)
        table, free, held, n_free = sim.table, sim.free, sim.held, sim.n_free
        owned = [table[r, i] for r in range(R) for i in range(held[r])]
        assert sorted(owned + free[:n_free].tolist()) == list(range(n_pages))  # every page in one place
        h_d, n_d = out["held"], out["n_free"]
        lens = [a + int(rng.integers(0, b + 1)) for a, b in zip(lens, rows)]
        lens = [min(a, 4 * page) for a in lens]
    assert int(err) == 0


@pytest.mark.parametrize("what", ["pages", "width", "rows", "parents", "negative", "tree", "held"])
def test_map_all_or_nothing(what):
    lens, rows, held = [5, 0, 9], [4, 2, 3], [2, 0, 3]
    page, N, n_free, parents, most = 4, 9, 6, None, None
    table = torch.arange(15, dtype=torch.int32, device="cuda").view(3, 5)
    if what == "pages":
        n_free = 0
    elif what == "width":
        lens[0] = 17
    elif what == "rows":
        N = 8
    elif what == "parents":
        parents, most = [-1] * 8, 4
    elif what == "negative":
        lens[1] = -1
    elif what == "tree":
        rows[0], N, parents, most = 65, 80, [-1] * 80, 64
        page = 64
    elif what == "held":
        held[2] = 6
    free = ints(list(range(20, 40)))
    err = err_word()
    before, stack = table.clone(), free.clone()
    out = dsp.page_map(ints(lens), ints(rows), table, ints(held), free, ints([n_free]), page=page, N=N,
                       parents=None if parents is None else ints(parents), max_rows=most, err=err)
    assert int(err) == _lib.ERR_RANGE
    assert torch.equal(table, before) and torch.equal(free, stack)
    assert out["held"].tolist() == held and int(out["n_free"]) == n_free
    assert out["row_start"].tolist() == [0] * 4 and out["slot"].tolist() == [-1] * N and out["pos"].tolist() == [0] * N


def test_map_bad_parent_is_reported():
    err = err_word()
    table, free = torch.full((1, 2), -1, dtype=torch.int32, device="cuda"), ints([0, 1])
    out = dsp.page_map(ints([3]), ints([4]), table, ints([0]), free, ints([2]), page=4, N=4,
                       parents=ints([-1, 0, 2, 1]), max_rows=4, err=err)
    assert int(err) == _lib.ERR_RANGE
    assert out["mask"].flatten().tolist() == [1, 3, 4, 11] and out["pos"].tolist() == [3, 4, 3, 5]


# ------------------------------------------------------------------ cache store
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,H,D,page", [(1, 1, 1, 1), (7, 3, 40, 5), (33, 8, 128, 16), (300, 2, 65, 32), (2, 1, 256, 64)])
def test_store(dtype, N, H, D, page):
    g = torch.Generator(device="cuda").manual_seed(N)
    n_pages = N // page + 3
    kc, vc = (torch.randn((n_pages, H, page, D), generator=g, device="cuda").to(dtype) for _ in range(2))
    fused = torch.randn((N, 3 * H + 1, D + 3), generator=g, device="cuda").to(dtype)
    k, v = fused[:, 1:1 + H, :D], fused[:, 1 + H:1 + 2 * H, :D]
    slot = torch.randperm(n_pages * page, generator=g, device="cuda")[:N].to(torch.int32)
    slot[N // 2] = -1
    want_k, want_v = kc.clone(), vc.clone()
    for i, s in enumerate(slot.tolist()):
        if s >= 0:
            want_k[s // page, :, s % page], want_v[s // page, :, s % page] = k[i], v[i]
    err = err_word()
    dsp.cache_store(k, v, slot, kc, vc, err=err)
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v) and int(err) == 0
    slot[0] = n_pages * page
    dsp.cache_store(k, v, slot, kc, vc, err=err)
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v) and int(err) == _lib.ERR_RANGE


# ------------------------------------------------------------------ attention
def make(lens, rows, Hq, H, D, page, dtype, seed=0, tree=False, extra=2, spread=1.0):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    N, R = sum(rows), len(rows)
    need = [-(-(a + b) // page) for a, b in zip(lens, rows)]
    n_pages = sum(need) + extra
    order = rng.permutation(n_pages)
    table = np.full((R, max(need) + 1), -1, np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    kc, vc = (torch.randn((n_pages, H, page, D), generator=g, device="cuda").to(dtype) for _ in range(2))
    q = (torch.randn((N, Hq + 2, D), generator=g, device="cuda") * spread).to(dtype)[:, 1:1 + Hq]
    s = dict(lens=lens, rows=rows, q=q, kc=kc, vc=vc, table=torch.from_numpy(table).cuda(), page=page,
             start=np.concatenate([[0], np.cumsum(rows)]).astype(int).tolist(), mask=None, scale=D ** -0.5)
    if tree:
        W = (max(rows) + 63) // 64
        s["mask"] = torch.from_numpy(words_of([b for n in rows for b in ancestors(tree_of(n, rng))], W)).cuda()
    return s


def call(s, **kw):
    err = err_word()
    out = dsp.tree_attention(s["q"], s["kc"], s["vc"], s["table"], ints(s["lens"]), ints(s["start"]), mask=s["mask"],
                             scale=s["scale"], max_rows=max(s["rows"]), err=err, **kw)
    return out, err


def expect(s):
    """(out, lse, ds, max|v|) per row and head in 64 bits; what a row does not see is not read."""
    q = s["q"].double()
    N, Hq, D = q.shape
    H = s["kc"].shape[1]
    out, lse = torch.zeros_like(q), torch.full((N, Hq), -INF, dtype=torch.float64, device="cuda")
    ds, vmax = torch.zeros((N, Hq), dtype=torch.float64, device="cuda"), torch.zeros((N, Hq), dtype=torch.float64, device="cuda")
    for r, (n_ctx, n) in enumerate(zip(s["lens"], s["rows"])):
        t = torch.arange(n_ctx + n, device="cuda")
        pg = s["table"][r].long()[t // s["page"]]
        k, v = (s[c][pg, :, t % s["page"]].double().transpose(0, 1) for c in ("kc", "vc"))
        for j in range(n):
            i = s["start"][r] + j
            if s["mask"] is None:
                seen = list(range(n_ctx + j + 1))
            else:
                w = [int(x) for x in s["mask"][i]]
                seen = list(range(n_ctx)) + [n_ctx + u for u in range(n) if (w[u // 64] >> (u % 64)) & 1]
            if not seen:
                continue
            kk, vv = (x[:, seen].repeat_interleave(Hq // H, 0) for x in (k, v))
            x = (kk @ q[i][:, :, None]).squeeze(-1) * s["scale"]
            lse[i] = torch.logsumexp(x, 1)
            out[i] = (torch.softmax(x, 1)[:, None] @ vv).squeeze(1)
            size = lambda x: x.abs().nan_to_num(0.0, 0.0, 0.0)  # noqa: E731  (of the finite values)
            ds[i] = ((size(kk) @ size(q[i])[:, :, None]).squeeze(-1).amax(1) * abs(s["scale"])) * D * 2.0 ** -24
            vmax[i] = size(vv).amax((1, 2))
    return out, lse, ds, vmax


def check(s, got, err, want=None):
    out, lse, ds, vmax = want or expect(s)
    assert int(err) == 0
    o, lg = got["out"].double(), got["lse"].double()
    n = max(a + b for a, b in zip(s["lens"], s["rows"]))
    fine = torch.isfinite(out)
    assert torch.equal(torch.isfinite(o), fine)
    assert torch.equal(o[~fine & ~out.isnan()], out[~fine & ~out.isnan()]) and torch.equal(o.isnan(), out.isnan())
    tol = ((2 * (ds + 1e-6) + 2.0 ** -24 * (n ** 0.5 + 64)) * vmax)[:, :, None].expand_as(out)
    if s["q"].dtype == torch.bfloat16:
        tol = tol + 2.0 ** -9 * vmax[:, :, None] + 2.0 ** -8 * out.abs()
    assert ((o - out).abs()[fine] <= tol[fine]).all(), float(((o - out).abs() / tol.clamp(min=1e-30))[fine].max())
    ok = torch.isfinite(lse)
    assert torch.equal(lg[~ok & ~lse.isnan()], lse[~ok & ~lse.isnan()]) and torch.equal(lg.isnan(), lse.isnan())
    assert ((lg - lse).abs()[ok] <= (ds + 1e-6 * (1 + lse.abs()))[ok]).all()


LAYOUTS = [(1, 1, 64, 16), (8, 2, 128, 16), (32, 8, 128, 32), (7, 1, 128, 8), (6, 3, 80, 48), (12, 4, 96, 64), (4, 4, 64, 128),
           (8, 8, 128, 256), (2, 1, 8, 16), (3, 1, 40, 5), (5, 5, 1, 3), (4, 2, 256, 16), (16, 2, 200, 7), (2, 2, 130, 16)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hq,H,D,page", LAYOUTS)
def test_attention_layouts(dtype, Hq, H, D, page):
    """Ragged chains: caches of none, one and many tokens, ends inside pages and tiles."""
    s = make([0, 1, 127, 128, 129, 63, 700, 0], [1, 5, 1, 3, 9, 2, 17, 4], Hq, H, D, page, dtype, seed=D + page)
    check(s, *call(s))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,ctx,G", [(1, 0, 4), (64, 100, 1), (65, 127, 2), (128, 300, 4), (256, 1000, 3), (200, 5, 8)])
def test_attention_trees(dtype, n, ctx, G):
    s = make([ctx, 2 * ctx + 3, ctx], [n, 7, max(1, n // 2)], 2 * G, 2, 64, 16, dtype, seed=n, tree=True)
    check(s, *call(s))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_long_chain(dtype):
    """A prompt in one call: more lines than a unit holds, every row a longer view."""
    s = make([0, 300], [401, 3], 4, 2, 128, 16, dtype, seed=3)
    check(s, *call(s))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,ctx", [(1, 20000), (3, 9000), (200, 50)])
def test_attention_split_and_packed(dtype, R, ctx):
    """One cache over many CTAs, and many caches in one."""
    rng = np.random.default_rng(R)
    lens = [int(rng.integers(ctx // 2, ctx + 1)) for _ in range(R)]
    s = make(lens, [int(rng.integers(1, 4)) for _ in range(R)], 8, 4, 128, 32, dtype, seed=R)
    check(s, *call(s))


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("lens,rows", [([3000, 10, 700, 0, 129, 5000], [1, 40, 64, 3, 65, 17]), ([0, 0, 0], [33, 1, 64]),
                                       ([20000, 127], [64, 32]), ([60] * 40, [34, 2, 64, 30] * 10)])
def test_attention_small_and_large_blocks(tree, lens, rows):
    """Requests whose rows fill one operand of the tensor cores beside ones that need two."""
    s = make(lens, rows, 8, 2, 128, 16, torch.bfloat16, seed=len(lens), tree=tree)
    check(s, *call(s))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("spread", [0.0, 30.0])
def test_attention_flat_and_peaked(dtype, spread):
    s = make([900, 40], [5, 2], 8, 2, 64, 16, dtype, seed=1, spread=spread)
    check(s, *call(s))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_requests_without_rows(dtype):
    s = make([50, 10, 0, 99], [0, 3, 0, 2], 4, 2, 64, 16, dtype)
    check(s, *call(s))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_empty_rows(dtype):
    """A mask that leaves nothing: zeros and -inf, whatever stands in the cache."""
    s = make([0, 0, 40], [6, 70, 5], 8, 2, 128, 16, dtype, tree=True)
    s["mask"][0] = 0
    s["mask"][3] = 0
    s["mask"][6 + 69] = 0
    s["mask"][6 + 70] = 0  # of the cached request: the cache alone
    want = expect(s)
    got, err = call(s)
    check(s, got, err, want)
    for i in (0, 3, 75):
        assert not got["out"][i].any() and (got["lse"][i] == -INF).all()
    s["vc"].fill_(float("nan"))
    got, _ = call(s)
    for i in (0, 3, 75):
        assert not got["out"][i].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("what", [float("nan"), INF, -INF])
@pytest.mark.parametrize("ctx,n,tree", [(37, 20, True), (120, 9, False), (0, 130, True), (128, 64, True), (500, 3, False)])
def test_attention_what_is_not_seen_has_no_influence(dtype, what, ctx, n, tree):
    """Stale slots and rows that others do not see hold infinities and NaN."""
    s = make([ctx, 11], [n, 2], 8, 2, 128, 16, dtype, seed=n, tree=tree, extra=3)
    bad = torch.ones(s["kc"].shape[0], s["page"], dtype=torch.bool, device="cuda")
    for r, (a, b) in enumerate(zip(s["lens"], s["rows"])):
        for t in range(a + b):
            bad[int(s["table"][r, t // s["page"]]), t % s["page"]] = False
    for c in ("kc", "vc"):
        s[c][bad[:, None, :].expand(s[c].shape[:3])] = what
    check(s, *call(s))
    # a row of the cycle itself: those that see it, and they alone, are touched
    t = ctx + n - 2 if n > 2 else ctx + 1
    pg, off = int(s["table"][0, t // s["page"]]), t % s["page"]
    s["vc"][pg, :, off, ::3] = what
    check(s, *call(s))
    s["kc"][pg, :, off] = what
    want = expect(s)
    got, err = call(s)
    seen = ~torch.isfinite(want[0]).all(-1) | ~torch.isfinite(want[1])
    for k, w in (("out", want[0]), ("lse", want[1])):
        assert torch.equal(torch.isfinite(got[k].double())[~seen], torch.isfinite(w)[~seen])
    keep = ~seen
    assert ((got["out"].double() - want[0]).abs()[keep] <= 0.05).all() and ((got["lse"].double() - want[1]).abs()[keep] <= 0.01).all()
    assert not torch.isfinite(got["lse"][seen & want[1].isnan()]).any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_offsets_beyond_32_bits(dtype):
    """A cache of more than 2^31 elements, its last pages in use."""
    H, page, D = 8, 64, 128
    n_pages = (1 << 31) // (H * page * D) + 40
    kc = torch.zeros((n_pages, H, page, D), dtype=dtype, device="cuda")
    vc = torch.zeros_like(kc)
    small = make([700, 300], [3, 9], 16, H, D, page, dtype, seed=5, extra=0)
    n = small["kc"].shape[0]
    kc[-n:], vc[-n:] = small["kc"], small["vc"]
    want = expect(small)
    s = dict(small, kc=kc, vc=vc, table=torch.where(small["table"] >= 0, small["table"] + n_pages - n, -1).int())
    check(s, *call(s), want)
    k = torch.randn((2, H, D), device="cuda").to(dtype)
    slot = ints([n_pages * page - 1, n_pages * page - page])
    dsp.cache_store(k, -k, slot, kc, vc)
    assert torch.equal(kc[-1, :, -1], k[0]) and torch.equal(vc[-1, :, 0], -k[1])


def test_attention_on_another_stream_and_in_a_graph():
    s = make([900, 40, 3], [5, 2, 1], 8, 2, 128, 16, torch.bfloat16, seed=1)
    want = expect(s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, err = call(s, stream=side)
    side.synchronize()
    check(s, got, err, want)
    lens, start, err = ints(s["lens"]), ints(s["start"]), err_word()
    ws = torch.empty(dsp.tree_attention_workspace_size(s["q"], s["kc"], s["vc"], s["table"], lens, start, max_rows=5),
                     dtype=torch.uint8, device="cuda")
    out = {"out": torch.zeros(s["q"].shape, dtype=s["q"].dtype, device="cuda"), "lse": torch.zeros(s["q"].shape[:2], device="cuda")}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsp.tree_attention(s["q"], s["kc"], s["vc"], s["table"], lens, start, max_rows=5, out=out, ws=ws, err=err)
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_device_side_errors(dtype):
    """Sizes and pages out of range are reported; the other requests' rows are right."""
    s = make([60, 30, 90], [3, 2, 4], 4, 2, 64, 16, dtype, seed=2)
    want = expect(s)
    for change in ("long", "negative", "page"):
        lens, table = list(s["lens"]), s["table"].clone()
        if change == "long":
            lens[1] = 10 ** 9
        elif change == "negative":
            lens[1] = -5
        else:
            table[1, 0] = 1 << 30
        err = err_word()
        got = dsp.tree_attention(s["q"], s["kc"], s["vc"], table, ints(lens), ints(s["start"]), scale=s["scale"], max_rows=4, err=err)
        assert int(err) == _lib.ERR_RANGE
        keep = [0, 1, 2, 5, 6, 7, 8]
        part = dict(s, q=s["q"][keep])
        check(part, {k: v[keep] for k, v in got.items()}, err_word(), tuple(w[keep] for w in want))


def test_attention_rows_beyond_the_batch_stay():
    s = make([60, 30], [3, 2], 4, 2, 64, 16, torch.bfloat16, seed=2)
    q = torch.cat([s["q"], s["q"]])
    out = {"out": torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda"), "lse": torch.full(q.shape[:2], 7.0, device="cuda")}
    dsp.tree_attention(q, s["kc"], s["vc"], s["table"], ints(s["lens"]), ints(s["start"]), scale=s["scale"], out=out)
    assert (out["out"][5:] == 7).all() and (out["lse"][5:] == 7).all()
    check(s, {k: v[:5] for k, v in out.items()}, err_word())


def test_attention_same_bits_again():
    s = make([9000, 40, 333], [5, 2, 1], 8, 2, 128, 16, torch.bfloat16, seed=1)
    a, _ = call(s)
    for _ in range(3):
        b, _ = call(s)
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [0.0, -0.25, 0.5])
def test_attention_scales(dtype, scale):
    s = make([300, 0, 77], [3, 2, 40], 8, 2, 64, 16, dtype, seed=3, tree=True)
    s["scale"] = scale
    check(s, *call(s))


def shifted(t):
    """The same values, contiguous, one element after an aligned address."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    out = flat[1:].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("what", ["q", "kc", "vc", "q_row", "q_head", "out"])
def test_attention_alignment(dtype, what):
    s = make([300, 0, 77], [3, 2, 40], 8, 2, 64, 16, dtype, seed=4)
    s["q"] = s["q"].contiguous()
    N, Hq, D = s["q"].shape
    kw = {}
    if what in ("q", "kc", "vc"):
        s[what] = shifted(s[what])
    elif what == "out":
        kw["out"] = {"out": shifted(s["q"]), "lse": torch.empty((N, Hq), device="cuda")}
    else:
        wide = torch.zeros((N, Hq * D + 1) if what == "q_row" else (N, Hq, D + 3), dtype=dtype, device="cuda")
        view = wide[:, :Hq * D].view(N, Hq, D) if what == "q_row" else wide[:, :, :D]
        view.copy_(s["q"])
        s["q"] = view
    got, err = call(s, **kw)
    check(s, got, err)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_rows_of_one_tensor(dtype):
    """Every row reads the same queries (a stride of zero)."""
    s = make([30, 150], [2, 3], 4, 2, 64, 16, dtype, seed=5)
    s["q"] = s["q"][:1].expand(5, -1, -1)
    check(s, *call(s))


def test_operators_between_other_work_in_a_graph():
    """A kernel waits for whatever stands before it, of this library or not, on its
    own stream or joined to it by an event; what stands after it sees its results."""
    lens, rows, page, V = [70, 0, 33], [3, 2, 4], 16, 777
    s = make(lens, rows, 4, 2, 64, page, torch.bfloat16, seed=6)
    want = expect(s)
    N, H, D = sum(rows), 2, 64
    n, held, free, n_free = ints(rows), ints([0] * 3), ints(list(range(40))), ints([40])
    lens_g, table = ints(lens), torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    k, v, q = (torch.empty_like(x) for x in (s["q"][:, :H].contiguous(), s["q"][:, :H].contiguous(), s["q"].contiguous()))
    start = s["start"]
    ctx_k, ctx_v = torch.zeros((40, H, page, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((40, H, page, D), dtype=torch.bfloat16, device="cuda")
    rows_k, rows_v = [], []
    for r in range(3):
        for t in range(lens[r], lens[r] + rows[r]):
            p = int(s["table"][r, t // page])
            rows_k.append(s["kc"][p, :, t % page])
            rows_v.append(s["vc"][p, :, t % page])
    rows_k, rows_v = torch.stack(rows_k), torch.stack(rows_v)
    T0 = torch.randn((N, V), device="cuda")
    T, err = torch.empty_like(T0), err_word()
    pres = torch.tensor([1.0, 2.0, 3.0], device="cuda")
    hist, hist_len = torch.zeros((3, 1), dtype=torch.int32, device="cuda"), ints([1, 1, 1])
    # the pages that the map will take hold the caches' tokens
    probe = dsp.page_map(lens_g, n, table.clone(), held, free.clone(), n_free, page=page, N=N)
    assert probe["row_start"].tolist() == start
    trial = table.clone()
    dsp.page_map(lens_g, n, trial, held, free.clone(), n_free, page=page, N=N)
    for r in range(3):
        for t in range(lens[r]):
            a, b = int(trial[r, t // page]), int(s["table"][r, t // page])
            ctx_k[a, :, t % page], ctx_v[a, :, t % page] = s["kc"][b, :, t % page], s["vc"][b, :, t % page]
    kc, vc = torch.empty_like(ctx_k), torch.empty_like(ctx_v)

    def cycle(side):
        here = torch.cuda.current_stream()
        kc.copy_(ctx_k)
        m = dsp.page_map(lens_g, n, table, held, free, n_free, page=page, N=N, err=err)
        fork = torch.cuda.Event()
        fork.record(here)
        with torch.cuda.stream(side):
            side.wait_event(fork)
            k.copy_(rows_k)
            v.copy_(rows_v)
            vc.copy_(ctx_v)
            q.copy_(s["q"])
            join = torch.cuda.Event()
            join.record(side)
        here.wait_event(join)
        dsp.cache_store(k, v, m["slot"], kc, vc, err=err)
        o = dsp.tree_attention(q, kc, vc, table, lens_g, m["row_start"], scale=s["scale"], max_rows=4, err=err)
        T.copy_(T0)
        z = dsp.logit_rules(T, m["row_start"], hist=hist, hist_len=hist_len, pres=pres, err=err)
        T.zero_()
        after = o["out"] * 1
        return o, z, after

    side = torch.cuda.Stream()
    rules = T0.clone()
    rules[:, 0] -= torch.repeat_interleave(pres, n.long())

    def right(o, z, after):
        check(s, o, err, want)
        assert torch.equal(z, rules) and torch.equal(after, o["out"])

    for _ in range(3):
        right(*cycle(side))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = cycle(side)
    for _ in range(3):
        for x in (kc, vc, k, v, q, T):
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        right(*got)


# ------------------------------------------------------------------ rules
def rules_case(R, most, V, dtype, seed, tree=False, hist=60, bias=6):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = rng.integers(0, most + 1, R).tolist()
    rows[0] = most
    N = sum(rows)
    s = dict(rows=rows, start=np.concatenate([[0], np.cumsum(rows)]).astype(int).tolist(), mask=None)
    s["T"] = (torch.randn((N, V), generator=g, device="cuda") * 4).to(dtype)
    some = rng.integers(0, V, 12)
    s["hist"] = np.where(rng.random((R, hist)) < 0.5, rng.choice(some, (R, hist)), rng.integers(0, V, (R, hist))).astype(np.int32)
    s["hist_len"] = rng.integers(0, hist + 1, R)
    s["prompt_len"] = np.array([rng.integers(0, n + 1) for n in s["hist_len"]])
    s["tok"] = rng.choice(some, N)
    s["rep"], s["freq"], s["pres"] = rng.uniform(0.8, 1.5, R), rng.uniform(-0.5, 1, R), rng.uniform(-0.5, 1, R)
    s["rep"][R // 2], s["freq"][R // 2], s["pres"][R // 2] = 1, 0, 0
    n_bias = rng.integers(0, bias + 1, R)
    s["bias_start"] = np.concatenate([[0], np.cumsum(n_bias)])
    s["bias_id"] = rng.choice(some, s["bias_start"][-1])
    s["bias_val"] = rng.uniform(-5, 5, s["bias_start"][-1])
    s["allow_row"] = np.array([-1 if rng.random() < 0.4 else rng.integers(0, 3) for _ in range(N)])
    s["allow"] = rng.random((3, V)) < np.array([0.02, 0.5, 0.0])[:, None]
    if tree:
        W = (most + 63) // 64
        s["mask"] = torch.from_numpy(words_of([b for n in rows for b in ancestors(tree_of(n, rng))], W)).cuda()
    return s


def rules_args(s):
    f = lambda v: torch.tensor(np.asarray(v), dtype=torch.float32, device="cuda")  # noqa: E731
    i = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")  # noqa: E731
    V = s["T"].shape[1]
    pad = np.pad(s["allow"], ((0, 0), (0, -V % 32))).reshape(s["allow"].shape[0], -1, 32)
    words = (pad.astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)
    return dict(tok=i(s["tok"]), mask=s["mask"], hist=i(s["hist"]), hist_len=i(s["hist_len"]), prompt_len=i(s["prompt_len"]),
                rep=f(s["rep"]), freq=f(s["freq"]), pres=f(s["pres"]), bias_start=i(s["bias_start"]), bias_id=i(s["bias_id"]),
                bias_val=f(s["bias_val"]), allow=torch.from_numpy(words).cuda(), allow_row=i(s["allow_row"]))


def rules_expect(s, off=()):
    """(out, sum of the terms' sizes) in 64 bits."""
    T = s["T"].double().cpu().numpy()
    out, size = T.copy(), np.abs(T)
    V = T.shape[1]
    for r, n in enumerate(s["rows"]):
        text = s["hist"][r, :s["hist_len"][r]] if "hist" not in off else np.zeros(0, int)
        np_ = s["prompt_len"][r] if "prompt_len" not in off else 0
        par = [np.float64(np.float32(s[k][r])) if k not in off else d for k, d in (("rep", 1.0), ("freq", 0.0), ("pres", 0.0))]
        base = np.bincount(text[np_:], minlength=V)[:V]
        prompt = np.bincount(text[:np_], minlength=V)[:V] > 0
        for j in range(n):
            i = s["start"][r] + j
            path = []
            if "tok" not in off:
                word = [int(w) for w in s["mask"][i]] if s["mask"] is not None else None
                path = [u for u in range(1, n) if (u <= j if word is None else (word[u // 64] >> (u % 64)) & 1)]
            c = base + np.bincount([s["tok"][s["start"][r] + u] for u in path], minlength=V)
            z = T[i]
            z = np.where((c > 0) | prompt, np.where(z > 0, z / par[0], z * par[0]), z) - par[1] * c - par[2] * (c > 0)
            size[i] += np.abs(z) + abs(par[1]) * c + abs(par[2])
            if "bias" not in off:
                for b in range(s["bias_start"][r], s["bias_start"][r + 1]):
                    z[s["bias_id"][b]] += np.float64(np.float32(s["bias_val"][b]))
                    size[i, s["bias_id"][b]] += abs(s["bias_val"][b])
            if "allow" not in off and s["allow_row"][i] >= 0:
                z = np.where(s["allow"][s["allow_row"][i]], z, -INF)
            out[i] = z
    return out, size


def rules_check(s, got, want):
    out, size = want
    g = got.double().cpu().numpy()
    assert np.array_equal(g == -INF, out == -INF)
    ok = np.isfinite(out)
    g, out, size = g[ok], out[ok], size[ok]
    tol = 6 * 2.0 ** -24 * size
    if s["T"].dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(out)
    assert (np.abs(g - out) <= tol).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,most,V,tree", [(1, 1, 1, False), (3, 5, 1024, False), (4, 9, 1001, True), (2, 70, 333, True),
                                           (9, 3, 8192, False), (5, 4, 20000, True), (2, 2, 32001, False), (40, 3, 8200, False)])
def test_rules(dtype, R, most, V, tree):
    s = rules_case(R, most, V, dtype, seed=V + R, tree=tree)
    err = err_word()
    args = rules_args(s)
    keep = s["T"].clone()
    got = dsp.logit_rules(s["T"], ints(s["start"]), **args, err=err)
    assert int(err) == 0 and torch.equal(s["T"], keep)
    want = rules_expect(s)
    rules_check(s, got, want)
    same = dsp.logit_rules(keep, ints(s["start"]), **args, out=keep)  # in place
    assert same is keep and torch.equal(keep, got)
    # rows that do not start on the boundaries of the output's
    n = s["T"].numel()
    odd = torch.empty(n + 1, dtype=dtype, device="cuda")[1:].view_as(s["T"])
    assert torch.equal(dsp.logit_rules(s["T"], ints(s["start"]), **args, out=odd), got)
    odd.copy_(s["T"])
    assert torch.equal(dsp.logit_rules(odd, ints(s["start"]), **args), got)


@pytest.mark.parametrize("off", [("hist",), ("prompt_len",), ("tok",), ("rep",), ("freq",), ("pres",), ("bias",), ("allow",),
                                 ("rep", "freq", "pres"), ("rep", "freq", "pres", "bias"), ("hist", "tok", "rep", "freq", "pres", "bias", "allow")])
def test_rules_left_out(off):
    s = rules_case(4, 4, 3000, torch.float32, seed=len(off))
    args = rules_args(s)
    gone = {"hist": ("hist", "hist_len", "prompt_len"), "bias": ("bias_start", "bias_id", "bias_val"), "allow": ("allow", "allow_row")}
    for k in off:
        for name in gone.get(k, (k,)):
            args[name] = None
    rules_check(s, dsp.logit_rules(s["T"], ints(s["start"]), **args), rules_expect(s, off))


def test_rules_long_bias_lists_and_texts():
    """More bias entries in a slice than the kernel keeps at hand, repeats among them."""
    s = rules_case(2, 3, 700, torch.float32, seed=3, hist=5000, bias=0)
    rng = np.random.default_rng(0)
    s["bias_start"] = np.array([0, 900, 905])
    s["bias_id"], s["bias_val"] = rng.integers(0, 700, 905), rng.uniform(-1, 1, 905)
    out, size = rules_expect(s)
    rules_check(s, dsp.logit_rules(s["T"], ints(s["start"]), **rules_args(s)), (out, size * 4))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [4096, 6001])
def test_rules_texts_of_many_tokens(dtype, V):
    """More said tokens in a slice than the kernel lists."""
    s = rules_case(3, 4, V, dtype, seed=V, hist=9000)
    s["hist_len"][:2] = 9000
    s["prompt_len"][:2] = 4000
    rules_check(s, dsp.logit_rules(s["T"], ints(s["start"]), **rules_args(s)), rules_expect(s))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [512, 1001])
@pytest.mark.parametrize("most,tree,bias", [(12, True, 60), (9, False, 200), (64, True, 40), (100, True, 30), (200, False, 9), (5, True, 700)])
def test_rules_many_biases_and_drafts(dtype, V, most, tree, bias):
    """Biases and drafted tokens all over a small vocabulary, some of them twice; more
    than a warp prepares, and rows beyond 64 bits."""
    s = rules_case(3, most, V, dtype, seed=V + most, tree=tree, hist=200, bias=bias)
    rng = np.random.default_rng(most)
    s["bias_id"] = rng.integers(0, V, s["bias_start"][-1])
    s["tok"] = rng.integers(0, V, len(s["tok"]))
    rules_check(s, dsp.logit_rules(s["T"], ints(s["start"]), **rules_args(s)), rules_expect(s))
    out = s["T"].clone()
    rules_check(s, dsp.logit_rules(out, ints(s["start"]), out=out, **rules_args(s)), rules_expect(s))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hist,shift", [(16383, 0), (16384, 0), (40001, 0), (16381, 3)])
def test_rules_long_texts(dtype, hist, shift):
    """One token said nearly all the time, next to others; rows of the text that do
    not start on 16 bytes."""
    s = rules_case(3, 4, 1500, dtype, seed=hist, hist=hist)
    s["hist"][:, 7:] = np.where(np.arange(hist - 7) % 97 == 0, s["hist"][:, 7:], 701)
    s["hist_len"][:], s["prompt_len"][:] = (hist, hist - 1, hist), (0, 5, 16001 if hist > 16001 else 9)
    s["freq"] *= 2.0 ** -10
    args = rules_args(s)
    if shift:
        flat = torch.zeros(3 * hist + shift, dtype=torch.int32, device="cuda")
        flat[shift:] = args["hist"].flatten()
        args["hist"] = flat[shift:].view(3, hist)
    rules_check(s, dsp.logit_rules(s["T"], ints(s["start"]), **args), rules_expect(s))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1024, 1023])
def test_rules_infinities_and_nan(dtype, V):
    """-inf and NaN logits stay themselves where allowed and are -inf where not."""
    s = rules_case(2, 3, V, dtype, seed=4)
    s["T"][:, ::3] = -INF
    s["T"][:, 1::5] = float("nan")
    s["T"][:, 2::7] = INF
    got = dsp.logit_rules(s["T"], ints(s["start"]), **rules_args(s)).double().cpu().numpy()
    T = s["T"].double().cpu().numpy()
    for i in range(T.shape[0]):
        m = s["allow"][s["allow_row"][i]] if s["allow_row"][i] >= 0 else np.ones(V, bool)
        assert (got[i][~m] == -INF).all()
        assert np.array_equal(np.isnan(got[i][m]), np.isnan(T[i][m]))
        inf = m & np.isinf(T[i])
        assert np.array_equal(got[i][inf], T[i][inf])


def test_rules_errors_are_reported():
    base = rules_case(3, 4, 500, torch.float32, seed=6)
    want = rules_expect(base)
    for name, at, value in (("hist_len", 1, 10 ** 6), ("prompt_len", 0, -1), ("allow_row", 0, 3), ("bias_start", 1, 10 ** 6), ("tok", 1, 500)):
        args = rules_args(base)
        args[name][at] = value
        err = err_word()
        got = dsp.logit_rules(base["T"], ints(base["start"]), **args, err=err)
        assert int(err) == _lib.ERR_RANGE, name
        last = base["start"][2]  # the third request is untouched
        rules_check(dict(base, T=base["T"][last:]), got[last:], (want[0][last:], want[1][last:]))
    args = rules_args(base)
    args["hist"][0, 0] = 500
    args["hist_len"][0] = 60
    err = err_word()
    dsp.logit_rules(base["T"], ints(base["start"]), **args, err=err)
    assert int(err) == _lib.ERR_RANGE
    err = err_word()
    out = torch.full_like(base["T"], 3.0)
    start = list(base["start"])
    start[-1] = base["T"].shape[0] + 1
    dsp.logit_rules(base["T"], ints(start), **rules_args(base), out=out, err=err)
    assert int(err) == _lib.ERR_RANGE and (out[start[2]:] == 3).all()


# ------------------------------------------------------------------ refusals of the binding
def test_binding_refuses():
    s = make([60, 30], [3, 2], 4, 2, 64, 16, torch.bfloat16)
    lens, start = ints(s["lens"]), ints(s["start"])
    ok = (s["q"], s["kc"], s["vc"], s["table"], lens, start)
    with pytest.raises(TypeError):
        dsp.tree_attention(s["q"].float(), *ok[1:])
    with pytest.raises(TypeError):
        dsp.tree_attention(*ok[:4], lens.long(), start)
    with pytest.raises(ValueError):
        dsp.tree_attention(s["q"].transpose(1, 2), *ok[1:])
    with pytest.raises(ValueError):
        dsp.tree_attention(s["q"], s["kc"].cpu(), *ok[2:])
    with pytest.raises(ValueError):
        dsp.tree_attention(*ok[:5], start[:-1])
    with pytest.raises(ValueError):
        dsp.tree_attention(*ok, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(dsp.DSparkError):
        dsp.tree_attention(s["q"][:, :3], *ok[1:])
    with pytest.raises(ValueError):
        dsp.cache_store(s["q"][:, :2], s["q"][:, :3], ints([0] * 5), s["kc"], s["vc"])
    held, n_free = ints([0, 0]), ints([4])
    with pytest.raises(dsp.DSparkError):
        dsp.page_map(lens, lens, s["table"], held, ints([0] * 4), n_free, page=16, N=4,
                     out={"held": held, "n_free": ints([0]), "row_start": start, "slot": ints([0] * 4), "pos": ints([0] * 4)})
    with pytest.raises(ValueError):
        dsp.page_map(lens, lens, s["table"], held, ints([0] * 4), n_free, page=16, N=4, parents=ints([0]))
    T = torch.zeros((5, 10), device="cuda")
    with pytest.raises(TypeError):
        dsp.logit_rules(T, start.long())
    with pytest.raises(dsp.DSparkError):
        dsp.logit_rules(T, start, hist=torch.zeros((2, 3), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        dsp.logit_rules(T, start, allow=torch.zeros((2, 3), dtype=torch.int32, device="cuda"), allow_row=ints([0] * 5))
