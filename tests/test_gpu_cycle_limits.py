"""The small server (cycle.py) at its limits: texts that fill up, a cache without
the pages, prompts and texts that do not fit."""
import pytest
import torch

from speculative_decoding_drafter_markov_gb300 import _lib as dsp
from speculative_decoding_drafter_markov_gb300 import cycle as C
from speculative_decoding_drafter_markov_gb300 import workloads as W
from test_gpu_cycle import TOL, whole_text_logits


def state(s):
    return {k: getattr(s, k).tolist() for k in ("hist", "hist_len", "lens", "anchor", "held", "n_free", "done")}


def consistent(s, R=6):
    """Every page in one place; the cache holds a live text but for its last token."""
    owned = [int(s.table[r, i]) for r in range(R) for i in range(int(s.held[r]))]
    pages = s.target.caches[0][0].shape[0]
    assert sorted(owned + s.free[:int(s.n_free)].tolist()) == list(range(pages))
    for r in range(R):
        n = int(s.hist_len[r])
        if not s.done[r]:
            assert int(s.lens[r]) == n - 1 and int(s.anchor[r]) == int(s.hist[r, n - 1])


def check_logits(s, o, before, R=6):
    """The live requests' logits of a cycle are the ones of their whole texts."""
    start, ell = o["row_start"].tolist(), o["ell"].tolist()
    for r in range(R):
        if before["done"][r]:
            continue
        n = before["hist_len"][r]
        text = before["hist"][r][:n] + o["x"][r, :ell[r]].tolist()
        want = whole_text_logits(s.target, text)[n - 1:]
        assert (o["T"][start[r]:start[r + 1]].float() - want).abs().max() < TOL


@pytest.mark.gpu
def test_texts_fill_up():
    """To the last token of every text and beyond: full texts stay, their pages are
    back, and the others go on."""
    full = 48
    s = C.small_server(seed=11, max_text=full, rules=dict(pres=torch.full((6,), 0.3, device="cuda")))
    prompts = s.hist_len.tolist()
    for c in range(full + 3):
        before = state(s)
        o = s.cycle()
        check_logits(s, o, before)
        after = state(s)
        assert int(s.err) == 0 and bool(o["ok"])
        for r in range(6):
            new, n = int(o["n_new"][r]), before["hist_len"][r]
            assert after["hist_len"][r] == n + new <= full and (new > 0) == (not before["done"][r])
            assert after["hist"][r][:n] == before["hist"][r][:n]
            assert after["hist"][r][n:n + new] == o["out_tokens"][r, :new].tolist()
            assert after["done"][r] == (n + new == full)
            if before["done"][r]:
                assert after["held"][r] == 1 and after["lens"][r] == 0
        consistent(s)
    assert min(prompts) >= 1 and all(after["done"]) and after["hist_len"] == [full] * 6


@pytest.mark.gpu
def test_a_cycle_without_pages_changes_nothing():
    """Until a request is finished and its pages are there."""
    probe = C.small_server(seed=13, page=4)
    start_pages = sum(probe.held.tolist())
    s = C.small_server(seed=13, page=4, n_pages=start_pages + 9)
    for c in range(40):
        before = state(s)
        o = s.cycle()
        if not bool(o["ok"]):
            break
        check_logits(s, o, before)
        assert int(s.err) == 0
        consistent(s)
    assert not bool(o["ok"]) and int(s.err) == dsp.ERR_RANGE and c > 0
    assert o["n_new"].tolist() == [0] * 6 and state(s) == before
    assert not bool(s.cycle()["ok"]) and state(s) == before
    s.err.zero_()
    s.finish(max(range(6), key=lambda r: before["lens"][r]))
    before = state(s)
    o = s.cycle()
    assert bool(o["ok"]) and int(s.err) == 0 and int(o["n_new"].sum()) >= 5
    check_logits(s, o, before)
    consistent(s)


@pytest.mark.parametrize("what,over", [("texts", dict(max_text=65)), ("prompts", dict(max_text=8)), ("pages", dict(n_pages=2))])
def test_what_does_not_fit_is_refused(what, over):
    """Before anything reaches a GPU."""
    wl = W.small("heavy", R=2, gamma=4, V=512, r=64, d=64)
    target = C.StandInTarget(512, n_pages=over.pop("n_pages", 64), max_len=64, device="cpu")
    with pytest.raises(ValueError, match=what):
        C.Server(wl, target, [list(range(9)), list(range(40))], **dict(dict(max_text=64), **over))
    with pytest.raises(ValueError, match="prompts"):
        C.Server(wl, C.StandInTarget(512, device="cpu"), [[1], []])
    with pytest.raises(ValueError, match="prompts"):
        C.Server(wl, C.StandInTarget(512, device="cpu"), [[1]])
