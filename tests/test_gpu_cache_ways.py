"""The ways into and out of the cache together, as a server runs them: batch map,
norms and rotation, writes in 16 and in 4 bits, attention; and the small server with a
target that uses them.

Tolerances: of the rotation as in test_gpu_rope.py; what is held in 4 bits is equal to
the format's definition applied to the keys that the rotation gave; of the attention as
in test_gpu_attention4.py (also for 16 bits: its weights are rounded by 2^-8 at most)."""
import numpy as np
import pytest
import torch

import cache4_plain as c4
import speculative_decoding_drafter_markov_gb300 as dsp
from speculative_decoding_drafter_markov_gb300 import cycle as C
from test_gpu_attention4 import check as check_attention
from test_gpu_cycle import TOL
from test_gpu_rope import expect as turned, freqs, near
from test_gpu_target import ancestors, err_word, ints, tree_of, words_of

pytestmark = pytest.mark.gpu


class Texts:
    """What the caches should hold, token by token, on the host's side."""

    def __init__(self, R):
        self.k, self.v = [[] for _ in range(R)], [[] for _ in range(R)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hq,H,D,page,tree,most", [(8, 2, 64, 16, False, 4), (8, 2, 128, 8, True, 9), (4, 4, 96, 24, False, 40)])
def test_cycles(dtype, Hq, H, D, page, tree, most):
    """Chained cycles: rows are mapped, turned, written both ways and attend; some are accepted."""
    rng = np.random.default_rng(D)
    g = torch.Generator(device="cuda").manual_seed(D)
    R, n_pages, width = 5, 120, 24
    lens = [0] * R
    table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
    free = torch.from_numpy(rng.permutation(n_pages).astype(np.int32)).cuda()
    held, n_free = ints([0] * R), ints([n_pages])
    caches = [torch.zeros((n_pages, H, page, D), dtype=dtype, device="cuda") for _ in range(2)]
    four = [dsp.cache4(n_pages, H, page, D) for _ in range(2)]
    weights = [(1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dtype) for _ in range(2)]
    freq, err = freqs(D), err_word()
    text16, text4 = Texts(R), Texts(R)
    for turn in range(4):
        rows = [60, 1, 33, 7, 90] if turn == 0 else rng.integers(1, most + 1, R).tolist()
        branches = tree and turn > 0
        N, top = sum(rows) + 3, max(rows)
        parents = [p for n in rows for p in tree_of(n, rng)] if branches else None
        m = dsp.page_map(ints(lens), ints(rows), table, held, free, n_free, page=page, N=N, parents=ints(parents) if branches else None,
                         max_rows=top, err=err)
        held, n_free = m["held"], m["n_free"]
        fused = torch.randn((N, Hq + 2 * H, D), generator=g, device="cuda").to(dtype)
        q, k, v = fused[:, :Hq], fused[:, Hq:Hq + H], fused[:, Hq + H:]
        norm = dict(q_weight=weights[0], k_weight=weights[1], err=err)
        on_the_way = dsp.rope_store(q, k, v, m["pos"], freq, slot=m["slot"], k_cache=caches[0], v_cache=caches[1], **norm)
        apart = dsp.rope_store(q, k, None, m["pos"], freq, **norm)
        n = sum(rows)
        assert torch.equal(on_the_way["q"][:n], apart["q"][:n])
        near(apart["q"][:n], *(x[:n] for x in turned(q, m["pos"], freq, weights[0], False)), D, True)
        near(apart["k"][:n], *(x[:n] for x in turned(k, m["pos"], freq, weights[1], False)), D, True)
        values = dsp.cache_store4(apart["k"], v, m["slot"], *four, values=True, err=err)
        for name, x in (("k", apart["k"]), ("v", v)):
            assert np.array_equal(values[name][:n].double().cpu().numpy(), c4.held(*c4.quantise(x[:n].double().cpu().numpy())))
        # every way of reading: the same case with either cache
        start = m["row_start"].tolist()
        mask = torch.from_numpy(words_of([b for a, c in zip(start, rows) for b in ancestors(parents[a:a + c])], (top + 63) // 64)).cuda() \
            if branches else None
        if branches:
            assert torch.equal(m["mask"][:n], mask)
        for text, tk, tv in ((text16, apart["k"], v), (text4, values["k"], values["v"])):
            # a cache of its own in the texts' order, to compare with
            P = max(-(-(a + b) // page) for a, b in zip(lens, rows))
            kc, vc = (torch.zeros((R * P, H, page, D), dtype=torch.float32, device="cuda") for _ in range(2))
            for r in range(R):
                for c, old, new in ((kc, text.k[r], tk), (vc, text.v[r], tv)):
                    all_rows = torch.cat([torch.stack(old).float() if old else new[:0].float(), new[start[r]:start[r + 1]].float()])
                    flat = c[r * P:(r + 1) * P].transpose(1, 2).reshape(P * page, H, D)
                    flat[:len(all_rows)] = all_rows
                    c[r * P:(r + 1) * P] = flat.view(P, page, H, D).transpose(1, 2)
            s = dict(lens=lens, rows=rows, q=apart["q"][:n], kc=kc, vc=vc, table=torch.arange(R * P, device="cuda", dtype=torch.int32).view(R, P),
                     page=page, start=start, mask=mask, scale=D ** -0.5)
            attend, c = (dsp.tree_attention, caches) if text is text16 else (dsp.tree_attention4, four)
            got = attend(apart["q"], *c, table, ints(lens), m["row_start"], mask=m.get("mask"), max_rows=top, err=err)
            check_attention(s, {x: y[:n] for x, y in got.items()}, err)
        # accepted: a chain's first rows (of a tree its first row alone, whose slot is its position's)
        for r in range(R):
            take = rows[r] if turn == 0 else 1 if branches else int(rng.integers(1, rows[r] + 1))
            for text, tk, tv in ((text16, apart["k"], v), (text4, values["k"], values["v"])):
                text.k[r] += list(tk[start[r]:start[r] + take])
                text.v[r] += list(tv[start[r]:start[r] + take])
            lens[r] += take
    assert int(err) == 0


def test_a_layer_in_a_graph():
    """Map, rotation, write and attention captured once and replayed on other rows."""
    R, Hq, H, D, page, n_pages = 3, 8, 2, 128, 16, 60
    g = torch.Generator(device="cuda").manual_seed(1)
    N = 12
    fused = torch.randn((N, Hq + 2 * H, D), generator=g, device="cuda").bfloat16()
    lens, rows, freq = ints([40, 0, 130]), ints([4, 3, 5]), freqs(D)
    table, held = torch.full((R, 12), -1, dtype=torch.int32, device="cuda"), ints([0] * R)
    free, n_free = torch.arange(n_pages, dtype=torch.int32, device="cuda"), ints([n_pages])
    four = [torch.randint(0, 250, (n_pages, H, page * D * 9 // 16), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
    err = err_word()

    def layer():
        m = dsp.page_map(lens, rows, table, held, free, n_free, page=page, N=N, err=err)
        t = dsp.rope_store(fused[:, :Hq], fused[:, Hq:Hq + H], None, m["pos"], freq, err=err)
        dsp.cache_store4(t["k"], fused[:, Hq + H:], m["slot"], *four, err=err)
        return dsp.tree_attention4(t["q"], *four, table, lens, m["row_start"], max_rows=5, err=err)

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer()
    first = None
    for change in (0, 1, 0):
        fused.copy_(fused if not change else torch.randn(fused.shape, generator=g, device="cuda"))
        before = [c.clone() for c in four]
        graph.replay()
        torch.cuda.synchronize()
        after = [c.clone() for c in four]
        for c, b in zip(four, before):
            c.copy_(b)
        want = layer()
        torch.cuda.synchronize()
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
        assert all(torch.equal(a, c) for a, c in zip(after, four))
        assert first is None or change == 0 or not torch.equal(got["out"], first)
        first = got["out"].clone()
    assert int(err) == 0


def whole_text_logits(t, text):
    """Logits after every token of `text` of a target with rotary positions, without a cache, in fp32."""
    n, G = len(text), t.Hq // t.H
    x = t.emb[text].float()
    pos = torch.arange(n, device=x.device)
    norm = lambda y: torch.nn.functional.rms_norm(y, y.shape[-1:])  # noqa: E731
    for qkv, proj, (qw, kw) in zip(t.qkv, t.proj, t.norms):
        q, k, v = (norm(x) @ qkv.float().T).view(n, -1, t.D).split([t.Hq, t.H, t.H], 1)
        q, k = (turned(y, pos, t.freq, w, False)[0].float().repeat_interleave(c, 1) for y, w, c in ((q, qw, 1), (k, kw, G)))
        s = torch.einsum("ihd,jhd->hij", q, k) * t.D ** -0.5
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device=x.device).triu(1), -float("inf"))
        x = x + torch.einsum("hij,jhd->ihd", s.softmax(-1), v.repeat_interleave(G, 1)).flatten(1) @ proj.float().T
    return norm(x) @ t.head.float().T


def test_temporaries_on_a_busy_stream():
    """What is passed with `stream` and let go at once is not handed out again before the stream has used it."""
    g = torch.Generator(device="cuda").manual_seed(9)
    H, D, page, N = 2, 64, 16, 33
    rand = lambda *n: torch.randn(n, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, k, v, freq = rand(N, 4, D), rand(N, H, D), rand(N, H, D), torch.rand(D // 2, generator=g, device="cuda")
    ints = lambda t: torch.as_tensor(t, dtype=torch.int32).cuda()  # noqa: E731
    side = torch.cuda.Stream()

    def run(stream):
        caches = [dsp.cache4(3, H, page, D) for _ in range(2)]
        torch.cuda.synchronize()
        if stream is not None:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(20_000_000)
        junk = []
        turned = dsp.rope_store(q.clone(), k.clone(), None, ints(range(N)), freq, stream=stream)
        junk += [torch.full((1 << i,), 3, dtype=torch.int32, device="cuda") for i in range(6, 13)]
        dsp.cache_store4(k.clone(), v.clone(), ints(range(N)), *caches, stream=stream)
        junk += [torch.full((1 << i,), 5, dtype=torch.int32, device="cuda") for i in range(6, 13)]
        got = dsp.tree_attention4(q.clone(), *caches, ints([[0, 1, 2]]), ints([0]), ints([0, N]), max_rows=N, stream=stream)
        junk += [torch.full((1 << i,), 7, dtype=torch.int32, device="cuda") for i in range(6, 13)]
        torch.cuda.synchronize()
        return turned["q"], turned["k"], *caches, got["out"], got["lse"]

    assert all(torch.equal(a, b) for a, b in zip(run(None), run(side)))


@pytest.mark.parametrize("D,page", [(64, 16), (128, 8)])
def test_server_with_rotary_positions(D, page):
    """As the server's own test: logits against the target over the whole text (its tolerance, for the same reason)."""
    s = C.small_server(seed=4, D=D, page=page, rotary=True)
    accepted = 0
    for _ in range(3):
        before, texts = s.hist_len.tolist(), s.hist.clone()
        o = s.cycle()
        x, start, ell = o["x"], o["row_start"].tolist(), o["ell"].tolist()
        for r in range(6):
            text = texts[r, :before[r]].long().tolist() + x[r, :ell[r]].long().tolist()
            want = whole_text_logits(s.target, text)[before[r] - 1:]
            assert (o["T"][start[r]:start[r + 1]].float() - want).abs().max() < TOL
        accepted += int(o["n_accept"].sum())
    assert int(s.err) == 0 and accepted > 0


class HeldInSixteen(C.StandInTarget):
    """The target over caches of 16 bits that hold what another's of 4 bits stand for."""

    def forward(self, tok, pos, held, table, lens, row_start, *, max_rows=1, err=None):
        x = self.emb[tok.long()]
        for i, ((kc, vc), qkv, proj) in enumerate(zip(self.caches, self.qkv, self.proj)):
            for c, four in ((kc, held[i][0]), (vc, held[i][1])):
                c.copy_(torch.from_numpy(np.nan_to_num(c4.values(four.cpu().numpy(), self.page, self.D))))
            rows = torch.matmul(torch.nn.functional.rms_norm(x, x.shape[-1:]), qkv.T).view(x.shape[0], -1, self.D)
            q = dsp.rope_store(rows[:, :self.Hq], None, None, pos, self.freq, q_weight=self.norms[i][0], err=err)["q"]
            out = dsp.tree_attention(q, kc, vc, table, lens, row_start, max_rows=max_rows, err=err)
            x = x + torch.matmul(out["out"].flatten(1), proj.T)
        return torch.matmul(torch.nn.functional.rms_norm(x, x.shape[-1:]), self.head.T)


@pytest.mark.parametrize("rows", [(3, 4, 1, 2, 4, 4), (1, 1, 1, 1, 1, 1), (30, 2, 5, 40, 1, 9)])
def test_target_with_caches_of_four_bits(rows):
    """The same weights over caches of 4 bits, and of 16 bits with the same values: the two attentions differ by
    their weights' rounding (2^-8 and 2^-11) and the queries of the second layer by roundings, which the tolerance of the
    logits, a dozen roundings of 2^-9, covers.  (Keys and values have to be the held ones of both layers: a code
    whose quotient lies within a bf16 rounding of a half, one of about fifty, would come out one step apart.)"""
    four, sixteen = C.StandInTarget(512, seed=5, rotary=True, bits=4), HeldInSixteen(512, seed=5, rotary=True)
    rng = np.random.default_rng(sum(rows))
    err = err_word()
    lens, held, n_free = ints([0] * 6), ints([0] * 6), ints([256])
    table, free = torch.full((6, 12), -1, dtype=torch.int32, device="cuda"), torch.arange(256, dtype=torch.int32, device="cuda")
    for turn in range(3):
        n = [30, 70, 1, 16, 90, 7] if turn == 0 else rows
        tok = ints(rng.integers(0, 512, sum(n)).tolist())
        m = dsp.page_map(lens, ints(n), table, held, free, n_free, page=16, N=sum(n), err=err)
        held, n_free = m["held"], m["n_free"]
        a = four.forward(tok, m["pos"], m["slot"], table, lens, m["row_start"], max_rows=max(n), err=err)
        b = sixteen.forward(tok, m["pos"], four.caches, table, lens, m["row_start"], max_rows=max(n), err=err)
        assert (a.float() - b.float()).abs().max() < TOL
        lens = lens + ints(n)
    assert int(err) == 0


def test_server_with_caches_of_four_bits():
    for rotary in (False, True):
        s = C.small_server(seed=6, rotary=rotary, bits=4)
        new = sum(int(s.cycle()["n_new"].sum()) for _ in range(4))
        assert int(s.err) == 0 and new >= 4 * 6
        assert s.target.caches[0][0].dtype == torch.uint8 and s.target.caches[0][0].any()
    with pytest.raises(ValueError):
        C.StandInTarget(512, bits=8)
