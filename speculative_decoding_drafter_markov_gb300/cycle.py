"""A decoding server in small: the drafter's cycle around a target model whose
pass runs on the paged-cache operators.

One cycle, all on the GPU and without a wait on the host: draft, schedule,
flattened tags, batch map (pages, slots, positions), the target's pass (per layer
cache writes and attention over the cache), the rules on its logits,
verification, and the bookkeeping of what was accepted.  A request is verified no
further than its text has room, and is done when that is full; a cycle for which
the cache has not the pages changes nothing.  The target is a stand-in with random
weights (embeddings, attention layers, a vocabulary projection); the drafter's
inputs are the synthetic ones of `workloads`.

    python -m speculative_decoding_drafter_markov_gb300.cycle
"""
from __future__ import annotations

import argparse
import math

import torch

from . import _lib as dsp
from . import workloads as W


class StandInTarget:
    """Embeddings, `layers` attention layers with residuals and a vocabulary
    projection, random weights; keys and values live in paged caches."""

    def __init__(self, V, *, layers=2, Hq=8, H=2, D=64, n_pages=256, page=16, max_len=4096, dtype=torch.bfloat16, device="cuda",
                 seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        dm = Hq * D
        rand = lambda *n: (torch.randn(n, generator=g, device=device) / math.sqrt(n[-1])).to(dtype)  # noqa: E731
        self.Hq, self.H, self.D, self.page = Hq, H, D, page
        self.emb = torch.randn((V, dm), generator=g, device=device).to(dtype)
        self.place = torch.randn((max_len, dm), generator=g, device=device).to(dtype)
        self.qkv = [rand((Hq + 2 * H) * D, dm) for _ in range(layers)]
        self.proj = [rand(dm, dm) for _ in range(layers)]
        self.head = rand(V, dm) * 4
        cache = lambda: torch.zeros((n_pages, H, page, D), dtype=dtype, device=device)  # noqa: E731
        self.caches = [(cache(), cache()) for _ in range(layers)]

    def forward(self, tok, pos, slot, table, lens, row_start, *, mask=None, max_rows=1, err=None):
        """Target logits [N, V] of rows with these tokens, positions and slots;
        their keys and values are in the caches afterwards."""
        x = self.emb[tok.long()] + self.place[pos.long()]
        for (kc, vc), qkv, proj in zip(self.caches, self.qkv, self.proj):
            rows = torch.matmul(torch.nn.functional.rms_norm(x, x.shape[-1:]), qkv.T).view(x.shape[0], -1, self.D)
            q, k, v = rows.split([self.Hq, self.H, self.H], 1)
            dsp.cache_store(k, v, slot, kc, vc, err=err)
            # rows beyond the batch are not written by the attention
            out = {"out": torch.zeros((x.shape[0], self.Hq, self.D), dtype=x.dtype, device=x.device)}
            dsp.tree_attention(q, kc, vc, table, lens, row_start, mask=mask, max_rows=max_rows, out=out, err=err)
            x = x + torch.matmul(out["out"].flatten(1), proj.T)
        return torch.matmul(torch.nn.functional.rms_norm(x, x.shape[-1:]), self.head.T)


class Server:
    """R requests decoded together, texts of up to `max_text` tokens; `rules` are the
    keyword arguments of dsp.logit_rules that do not change from cycle to cycle."""

    def __init__(self, wl, target, prompts, *, seed=0, max_text=512, rules=None):
        dev = target.emb.device
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
        self.wl, self.target, self.seed, self.cycles = wl, target, seed, 0
        self.rules = rules or {}
        n_pages = target.caches[0][0].shape[0]
        R, width = wl.R, (max_text + wl.gamma) // target.page + 2
        if max_text > target.place.shape[0]:
            raise ValueError(f"texts of up to {max_text} tokens, above the target's {target.place.shape[0]}")
        if len(prompts) != R or not all(1 <= len(p) <= max_text for p in prompts):
            raise ValueError(f"{R} prompts of 1 to {max_text} tokens are needed")
        need = sum(-(-(len(p) - 1) // target.page) for p in prompts)
        if need > n_pages:
            raise ValueError(f"the prompts take {need} pages, the cache has {n_pages}")
        self.table = torch.full((R, width), -1, dtype=torch.int32, device=dev)
        self.held, self.free, self.n_free = i32([0] * R), torch.arange(n_pages, dtype=torch.int32, device=dev), i32([n_pages])
        self.lens = i32([0] * R)
        self.err = i32([0])
        self.hist = torch.zeros((R, max_text), dtype=torch.int32, device=dev)
        for r, p in enumerate(prompts):
            self.hist[r, :len(p)] = i32(p)
        self.hist_len = i32([len(p) for p in prompts])
        self.prompt_len = self.hist_len.clone()
        self.K = [i32([-1]), i32([-1])]
        B_min, _ = wl.B_range
        self.sps, self.B_min = torch.as_tensor(W.sps_table(wl), device=dev), B_min
        # all but a prompt's last token go into the caches now; the last is the anchor
        tok = [t for p in prompts for t in p[:-1]]
        rows = i32([len(p) - 1 for p in prompts])
        if tok:
            self.pass_of(i32(tok), rows, len(tok), max(len(p) for p in prompts))
        self.lens = rows
        self.anchor = i32([p[-1] for p in prompts])
        self.done = self.hist_len >= max_text

    def finish(self, r):
        """Request r is done: its pages go back in the next cycle, but for the one of an
        idle row (every cycle has a row of every request), and it gets no more tokens."""
        self.done[r] = True
        self.lens[r] = 0

    def pass_of(self, tok, rows, N, max_rows, parents=None):
        """Reserve pages for `rows` new rows per request and run the target on them."""
        m = dsp.page_map(self.lens, rows, self.table, self.held, self.free, self.n_free, page=self.target.page, N=N,
                         parents=parents, max_rows=max_rows, err=self.err)
        self.held, self.n_free = m["held"], m["n_free"]
        T = self.target.forward(tok, m["pos"], m["slot"], self.table, self.lens, m["row_start"], mask=m.get("mask"),
                                max_rows=max_rows, err=self.err)
        return T, m

    def cycle(self):
        """One decoding cycle.  Returns the drafted tokens, the verified lengths, the
        stand-in's logits T, the logits that it makes of them before and after the
        rules, and the outcome: "n_new" tokens of `out_tokens` are new text, none of a
        request that is done, and none at all where "ok" is false: the cache had not the
        pages (the error word says so), and the server stands where it stood."""
        wl, err = self.wl, self.err
        inp = W.draft_inputs(wl, seed=self.seed + self.cycles, device=self.anchor.device)
        key = dict(seed=self.seed, cycle=self.cycles, err=err)
        d = dsp.draft_markov(inp["U"], inp["h"], inp["W1"], inp["W2t"], inp["w"], self.anchor, **key)
        mode = dsp.SCHED_ASYNC if wl.sched == "async" else dsp.SCHED_SYNC
        s = dsp.schedule(d["c"], self.sps, self.B_min, mode=mode, K_in=self.K[0], err=err)
        self.K = [self.K[1], s["K_out"]]
        room = torch.where(self.done, 0, self.hist.shape[1] - self.hist_len)  # tokens
        ell = torch.minimum(s["ell"], (room - 1).clamp(min=0)).to(torch.int32)
        tags, N = dsp.build_tags(ell, wl.gamma, err=err)
        req, at = tags[:, 0].long().clamp(0, wl.R - 1), tags[:, 1].long().clamp(0, wl.gamma)
        used = torch.arange(tags.shape[0], device=tags.device) < N
        req, at = torch.where(used, req, 0), torch.where(used, at, 0)
        tok = torch.where(at == 0, self.anchor[req], d["x"][req, (at - 1).clamp(min=0)])
        rows = ell + 1
        T, m = self.pass_of(tok, rows, tags.shape[0], wl.gamma + 1)
        # a drafter that knows something of its target: the stand-in's logits move around
        # the drafter's base logits
        base = torch.cat([inp["U"], inp["U_bonus"][:, None]], 1)
        logits = (T.float() * 0.25 + base[req, at].float()).to(T.dtype)
        ruled = dsp.logit_rules(logits, m["row_start"], tok=tok, hist=self.hist, hist_len=self.hist_len, prompt_len=self.prompt_len,
                                out=torch.zeros_like(logits), err=err, **self.rules)
        v = dsp.verify(ruled, tags, self.anchor, d["x"], d["logq"], d["lse"], inp["U"], inp["W1"], inp["W2t"], N_dev=N, **key)
        # the anchor and the accepted tokens stay in the caches; they and the target's
        # own token are text.  (A map that failed has no rows; else there is one at least.)
        ok = m["row_start"][-1] > 0
        out, n = v["out_tokens"], torch.where(ok & ~self.done, v["n_accept"] + 1, 0)
        col = torch.arange(wl.gamma + 1, device=out.device)
        place = torch.where(col < n[:, None], self.hist_len[:, None] + col, self.hist.shape[1])
        pad = torch.nn.functional.pad(self.hist, (0, 1))  # where the other columns go
        self.hist = pad.scatter(1, place.long(), out)[:, :-1].contiguous()
        self.hist_len = self.hist_len + n
        self.done = self.done | (self.hist_len >= self.hist.shape[1])
        self.lens = torch.where(self.done, 0, self.lens + n)
        self.anchor = torch.where(n > 0, v["next_anchor"], self.anchor)
        self.cycles += 1
        return {"x": d["x"], "ell": ell, "row_start": m["row_start"], "T": T, "logits": logits,
                "ruled": ruled, "n_new": n, "ok": ok, **v}


def small_server(seed=0, *, R=6, gamma=4, V=2048, max_text=512, rules=None, **target):
    """A server of random prompts, small enough to run anywhere; with a cache that holds
    all texts unless `n_pages` says otherwise."""
    wl = W.small("heavy", R=R, gamma=gamma, V=V, r=64, d=64)
    g = torch.Generator().manual_seed(seed)
    prompts = [torch.randint(0, V, (int(torch.randint(1, 40, (1,), generator=g)),), generator=g).tolist() for _ in range(R)]
    target.setdefault("n_pages", max(256, R * ((max_text + gamma) // target.get("page", 16) + 1)))
    return Server(wl, StandInTarget(V, seed=seed, **target), prompts, seed=seed, max_text=max_text, rules=rules)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--cycles", type=int, default=8)
    ap.add_argument("--requests", type=int, default=6)
    a = ap.parse_args()
    R = a.requests
    per = lambda v: torch.full((R,), v, device="cuda")  # noqa: E731
    s = small_server(R=R, rules=dict(rep=per(1.2), freq=per(0.1), pres=per(0.0)))
    for c in range(a.cycles):
        o = s.cycle()
        print(f"cycle {c}: verified {int(o['ell'].sum())} drafted tokens, new tokens {int(o['n_new'].sum())}, "
              f"done {int(s.done.sum())}, pages free {int(s.n_free)}")
    assert int(s.err) == 0, f"device error {int(s.err)}"
    for r in range(R):
        n, p = int(s.hist_len[r]), int(s.prompt_len[r])
        print(f"request {r}: {n - p} tokens after a prompt of {p}: {s.hist[r, p:n].tolist()}")


if __name__ == "__main__":
    main()
