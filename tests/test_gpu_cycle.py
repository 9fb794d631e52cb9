"""The small server (cycle.py): the operators together, as a server uses them.

Every cycle's target logits from the paged caches are compared with the target
run over the whole text without a cache, in fp32; the ruled logits with the rules
of that text; a tree of candidates with its chains run one by one; and the pages
are all accounted for.

Tolerance of the logits: both sides run the same weights in bf16 and differ by
the rounding of activations (2^-9 each) through two layers and the projection,
a dozen roundings that add up like independent errors, on logits of size 4: 12^(1/2) 2^-9 4
= 0.03 typical; the largest of the thousands compared stays within six of that, 0.2.
"""
import numpy as np
import pytest
import torch

from speculative_decoding_drafter_markov_gb300 import _lib as dsp
from speculative_decoding_drafter_markov_gb300 import cycle as C

pytestmark = pytest.mark.gpu
TOL = 0.2


def whole_text_logits(t, text):
    """Logits after every token of `text`, without a cache, in fp32."""
    n, G = len(text), t.Hq // t.H
    x = (t.emb[text] + t.place[:n]).float()
    norm = lambda y: torch.nn.functional.rms_norm(y, y.shape[-1:])  # noqa: E731
    for qkv, proj in zip(t.qkv, t.proj):
        q, k, v = (norm(x) @ qkv.float().T).view(n, -1, t.D).split([t.Hq, t.H, t.H], 1)
        k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
        s = torch.einsum("ihd,jhd->hij", q, k) * t.D ** -0.5
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device=x.device).triu(1), -float("inf"))
        x = x + torch.einsum("hij,jhd->ihd", s.softmax(-1), v).flatten(1) @ proj.float().T
    return norm(x) @ t.head.float().T


@pytest.mark.parametrize("D,page", [(64, 16), (128, 8)])
def test_cycles_match_the_whole_text(D, page):
    per = lambda v: torch.full((6,), v, device="cuda")  # noqa: E731
    s = C.small_server(seed=3, rules=dict(rep=per(1.3), freq=per(0.2), pres=per(0.1)), D=D, page=page)
    accepted = 0
    for _ in range(4):
        before, texts = s.hist_len.tolist(), s.hist.clone()
        o = s.cycle()
        x, start, ell = o["x"], o["row_start"].tolist(), o["ell"].tolist()
        for r in range(6):
            n = before[r]
            text = texts[r, :n].long().tolist() + x[r, :ell[r]].long().tolist()
            want = whole_text_logits(s.target, text)[n - 1:]
            got = o["T"][start[r]:start[r + 1]].float()
            assert (got - want).abs().max() < TOL
            # the rules of the text and of the drafted tokens so far, from the logits themselves
            p = int(s.prompt_len[r])
            for j in range(ell[r] + 1):
                count = np.bincount(text[p:n + j], minlength=2048)
                said = np.bincount(text[:n + j], minlength=2048) > 0
                z = o["logits"][start[r] + j].float().cpu().numpy().astype(np.float64)
                z = np.where(said, np.where(z > 0, z / 1.3, z * 1.3), z) - 0.2 * count - 0.1 * (count > 0)
                ruled = o["ruled"][start[r] + j].float().cpu().numpy()
                assert np.all(np.abs(ruled - z) <= 2.0 ** -8 * np.abs(z) + 1e-5)
            # what came out is text now
            k = int(o["n_accept"][r]) + 1
            accepted += k - 1
            assert s.hist[r, n:n + k].tolist() == o["out_tokens"][r, :k].tolist()
            assert int(s.hist_len[r]) == n + k and int(s.lens[r]) == n + k - 1
        owned = [int(s.table[r, i]) for r in range(6) for i in range(int(s.held[r]))]
        pages = s.target.caches[0][0].shape[0]
        assert sorted(owned + s.free[:int(s.n_free)].tolist()) == list(range(pages))
    assert int(s.err) == 0 and accepted > 0


def test_grammar_keeps_the_output_inside():
    """Only allowed tokens come out of the verification."""
    allow = torch.zeros(2048, dtype=torch.bool)
    allow[torch.randperm(2048, generator=torch.Generator().manual_seed(1))[:20]] = True
    words = (allow.view(-1, 32).long() << torch.arange(32)).sum(-1).to(torch.uint32).view(torch.int32)
    rows = 6 * 5
    s = C.small_server(seed=5, rules=dict(allow=words[None].contiguous().cuda(), allow_row=torch.zeros(rows, dtype=torch.int32, device="cuda")))
    for _ in range(3):
        o = s.cycle()
        out = o["out_tokens"][o["out_tokens"] >= 0].long().cpu()
        assert allow[out].all()
    assert int(s.err) == 0


def test_tree_of_candidates_matches_its_chains():
    """Candidates of every request as one tree, and each branch as a chain of its own."""
    trees = [[-1, 0, 0, 1, 1, 2, 5], [-1, 0, 1, 2], [-1], [-1, 0, 0, 0, 2, 4, 4, 6], [-1, 0], [-1, 0, 1, 1]]
    V = 2048
    s = C.small_server(seed=7)
    g = torch.Generator().manual_seed(2)
    tok = [torch.randint(0, V, (len(t),), generator=g).tolist() for t in trees]
    for r, t in enumerate(tok):
        t[0] = int(s.anchor[r])
    flat = lambda v: torch.tensor([y for x in v for y in x], dtype=torch.int32, device="cuda")  # noqa: E731
    rows = torch.tensor([len(t) for t in trees], dtype=torch.int32, device="cuda")
    N = sum(map(len, trees))
    T, m = s.pass_of(flat(tok), rows, N, 8, parents=flat(trees))
    assert int(s.err) == 0
    start = m["row_start"].tolist()
    for r, t in enumerate(trees):
        text = s.hist[r, :int(s.hist_len[r])].long().tolist()[:-1]
        for j in range(len(t)):
            path, at = [], j
            while at >= 0:
                path.append(tok[r][at])
                at = t[at]
            want = whole_text_logits(s.target, text + path[::-1])[-1]
            assert (T[start[r] + j].float() - want).abs().max() < TOL
            assert int(m["pos"][start[r] + j]) == len(text) + len(path) - 1


def test_requests_come_and_go():
    """A finished request gives its pages back in the next map."""
    s = C.small_server(seed=9)
    s.cycle()
    zero = torch.zeros(6, dtype=torch.int32, device="cuda")
    lens = s.lens.clone()
    lens[2] = 0
    m = dsp.page_map(lens, zero, s.table, s.held, s.free, s.n_free, page=s.target.page, N=0, err=s.err)
    page = s.target.page
    assert m["held"].tolist() == [-(-n // page) for n in lens.tolist()] and int(m["held"][2]) == 0
    pages = s.target.caches[0][0].shape[0]
    assert int(m["n_free"]) == pages - sum(m["held"].tolist()) and int(s.err) == 0
