"""Cases of the target-pass operators: batch maps over a paged cache, the cache
writes, attention of drafted rows over the cache, and the logit rules.

One decoding cycle of a server drafts a few tokens per request (a chain, or a
tree of candidates), asks the target model for the logits of every drafted row
and verifies them.  Between the draft and the verification the server

* reserves pages of the key-value cache for the new rows (``page_map``),
* writes the rows' keys and values (``cache_store``),
* lets every row attend to its request's cache and to its own ancestors among
  the drafted rows (``tree_attention``), once per layer, and
* applies repetition penalties, biases and grammar masks to the target's logits
  (``logit_rules``).

``run`` computes a case in plain torch operations, or, with ``own`` set, by the
library's entry points.  ``exact`` computes it from the definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
INF = float("inf")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest call: four requests drafting a chain of four (the tiny workload), where latency counts
        dict(name="map_tiny", op="map", R=4, ctx=1000, rows=5, page=16, tree=False, even=False),
        # the prod workload's batch of 512 requests, each with a tree of up to 64 candidates, over 32K-token caches
        dict(name="map_tree", op="map", R=512, ctx=32768, rows=64, page=16, tree=True, even=False),
        # admission of 96 prompts, short and long, in one call
        dict(name="map_prompts", op="map", R=96, ctx=0, rows=32768, page=64, tree=False, even=False),
        # one layer's write of a qwen4b cycle: 64 requests, up to 9 rows each, 8 heads of 128
        dict(name="store_cycle", op="store", R=64, ctx=8192, rows=9, page=16, Hq=32, H=8, D=128, dtype="bf16"),
        # one layer's write of a batch of prompts, out of the fused query-key-value projection
        dict(name="store_prompts", op="store", R=24, ctx=0, rows=8192, page=64, Hq=32, H=8, D=128, dtype="bf16"),
        # plain decoding of a single request: one row
        dict(name="attn_single", op="attn", R=1, ctx=2047, rows=1, page=16, Hq=32, H=8, D=128, dtype="bf16", tree=False),
        # the tiny workload's precision: a few requests in 32 bits, chains of up to five rows
        dict(name="attn_f32", op="attn", R=4, ctx=1500, rows=5, page=16, Hq=8, H=4, D=64, dtype="f32", tree=False),
        # a qwen4b cycle: 64 requests with ragged caches and chains of up to 9 rows
        dict(name="attn_chain", op="attn", R=64, ctx=8192, rows=9, page=16, Hq=32, H=8, D=128, dtype="bf16", tree=False),
        # trees of up to 64 candidates over 16K-token caches
        dict(name="attn_tree", op="attn", R=16, ctx=16384, rows=64, page=32, Hq=32, H=8, D=128, dtype="bf16", tree=True),
        # few requests with very long caches, chains of up to 17 rows
        dict(name="attn_long", op="attn", R=8, ctx=131072, rows=17, page=64, Hq=32, H=8, D=128, dtype="bf16", tree=False),
        # the tiny workload's logits: 32 bits, a small vocabulary
        dict(name="rules_tiny", op="rules", R=4, rows=5, V=1024, hist=500, bias=8, dtype="f32", tree=False),
        # a prod cycle: 512 requests, up to 9 verified rows each, every rule in use
        dict(name="rules_prod", op="rules", R=512, rows=9, V=129280, hist=8192, bias=32, dtype="bf16", tree=False),
    ]


def log_int(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["map", "store", "attn", "attn", "attn", "rules"])
    page = rng.choice([8, 16, 16, 32, 48, 64, 128])
    if op == "map":
        if rng.random() < 0.3:
            return dict(op="map", R=log_int(rng, 1, 96), ctx=0, rows=log_int(rng, 16, 32768), page=page, tree=False, even=False)
        return dict(op="map", R=log_int(rng, 1, 512), ctx=log_int(rng, 1, 32768), rows=log_int(rng, 1, 64), page=page,
                    tree=rng.random() < 0.5, even=rng.random() < 0.3)
    if op == "rules":
        R = log_int(rng, 1, 512)
        return dict(op="rules", R=R, rows=log_int(rng, 1, 17), V=log_int(rng, 1000, 151936 if R <= 256 else 65536),
                    hist=log_int(rng, 1, 16384), bias=rng.choice([0, 5, 64]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    tree=rng.random() < 0.3)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    G = rng.choice([1, 2, 3, 4, 7, 8])
    H = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128, 128, 128, 80, 96])
    c = dict(op=op, R=log_int(rng, 1, 128), page=page, Hq=G * H, H=H, D=D, dtype=dtype)
    if op == "store":
        return dict(c, ctx=log_int(rng, 1, 4096), rows=log_int(rng, 1, 1024))
    # tokens of all caches together: at most half of attn_long's, an eighth in 32 bits
    most = (524288 if dtype == "bf16" else 131072) // c["R"]
    return dict(c, ctx=log_int(rng, 1, min(131072, most)), rows=log_int(rng, 1, 64 if c["R"] <= 32 else 17), tree=rng.random() < 0.4)


def lens_of(case):
    """Cache lengths before the cycle and new rows of every request: whole numbers that the case alone gives."""
    rng = random.Random(case["R"] * 7919 + case.get("ctx", 0) * 31 + case["rows"])
    R, ctx, rows = case["R"], case.get("ctx", case.get("hist", 0)), case["rows"]
    if case.get("even"):
        return [ctx] * R, [rows] * R
    lens = [ctx] + [log_int(rng, max(1, ctx // 16), ctx) if ctx else 0 for _ in range(R - 1)]
    new = [rows] + [log_int(rng, 1, rows) if rows > 64 else rng.randint(1, rows) for _ in range(R - 1)]
    return lens, new


# ------------------------------------------------------------------ inputs
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def ints(v):
    return torch.tensor(v, dtype=torch.int32).to(DEV)


def trees(new, rng):
    """Parents of every row within its request: -1 for the first, else a recent earlier row."""
    return [-1 if j == 0 else rng.randint(max(0, j - 8), j - 1) for n in new for j in range(n)]


def mask_words(new, parents, W):
    """[N, W] 64-bit words: bit j of row i is set where row j of its request is row i or one of its ancestors."""
    out, at = np.zeros((len(parents), W), np.uint64), 0
    for n in new:
        seen = []
        for j in range(n):
            p = parents[at + j]
            seen.append((seen[p] if p >= 0 else 0) | (1 << j))
            for w in range(W):
                out[at + j, w] = (seen[j] >> (64 * w)) & 0xFFFFFFFFFFFFFFFF
        at += n
    return out


def prepare(case, seed):
    rng = random.Random(seed * 1000003 + 17)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    lens, new = lens_of(case)
    both = list(zip(lens, new))
    rng.shuffle(both)
    lens, new = [a for a, _ in both], [b for _, b in both]
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s = dict(op=case["op"], N=start[-1], max_rows=max(new), lens=ints(lens), new=ints(new), row_start=ints(start), R=len(new),
             W=(max(new) + 63) // 64, err=torch.zeros(1, dtype=torch.int32, device=DEV), mask=None)
    parents = trees(new, rng) if case.get("tree") else None
    if case["op"] == "rules":
        if parents:
            s["mask"] = torch.from_numpy(mask_words(new, parents, s["W"]).view(np.int64)).to(DEV)
        return prepare_rules(case, s, lens, rng, gen)
    P = s["page"] = case["page"]
    need = [(a + b + P - 1) // P for a, b in zip(lens, new)]
    total, width = sum(need), max(need) + 2
    n_pages = s["n_pages"] = total + total // 8 + 2 * len(new) + 1
    order = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    if case["op"] == "map":
        # after the last cycle a request holds the pages of its old draft: one more, one fewer, or all it needs
        held = [min(width, max((a + P - 1) // P, n + rng.randint(-1, 1))) for a, n in zip(lens, need)]
        s.update(parents=ints(parents) if parents else None, held=ints(held), cap=s["N"] + 7)
        table, at = np.full((len(held), width), -1, np.int32), 0
        own_pages = order.cpu().numpy()
        for r, h in enumerate(held):
            table[r, :h] = own_pages[at:at + h]
            at += h
        free = np.full(n_pages, -1, np.int32)
        free[:n_pages - at] = own_pages[at:]
        s.update(table=torch.from_numpy(table).to(DEV), free=torch.from_numpy(free).to(DEV), n_free=ints([n_pages - at]))
        return s
    H, D, dt = case["H"], case["D"], TYPES[case["dtype"]]
    cols = torch.arange(width, device=DEV)
    used = cols[None, :] < ints(need)[:, None]
    table = torch.full((len(new), width), -1, dtype=torch.int32, device=DEV)
    table[used] = order[:total]
    fused = torch.randn((s["N"], (case["Hq"] + 2 * H) * D), generator=gen, device=DEV, dtype=torch.float32).to(dt)
    heads = fused.view(s["N"], case["Hq"] + 2 * H, D)
    k_cache = torch.randn((n_pages, H, P, D), generator=gen, device=DEV, dtype=dt)
    v_cache = torch.randn((n_pages, H, P, D), generator=gen, device=DEV, dtype=dt)
    s.update(table=table, k_cache=k_cache, v_cache=v_cache, q=heads[:, :case["Hq"]], k=heads[:, case["Hq"]:case["Hq"] + H],
             v=heads[:, case["Hq"] + H:], scale=1.0 / math.sqrt(D))
    if case["op"] == "store":
        req, at = rows_of(s)
        place = s["lens"].long()[req] + at
        s["slot"] = (table.long()[req, place // P] * P + place % P).to(torch.int32)
    elif parents:
        s["mask"] = torch.from_numpy(mask_words(new, parents, s["W"]).view(np.int64)).to(DEV)
    return s


def prepare_rules(case, s, lens, rng, gen):
    R, N, V, dt = case["R"], s["N"], case["V"], TYPES[case["dtype"]]
    s["T"] = (torch.randn((N, V), generator=gen, device=DEV) * 3.0).to(dt)
    # few tokens make up most of a text: squares of even numbers
    text = lambda *n: (torch.rand(n, generator=gen, device=DEV).square() * V).to(torch.int32).clamp_(max=V - 1)  # noqa: E731
    s["hist"], s["tok"] = text(R, case["hist"]), text(N)
    s["hist_len"] = ints(lens)
    s["prompt_len"] = ints([rng.randint(0, n) for n in lens])
    pick = lambda off, lo, hi: [off if rng.random() < 0.25 else rng.uniform(lo, hi) for _ in range(R)]  # noqa: E731
    for name, v in (("rep", pick(1.0, 1.05, 1.4)), ("freq", pick(0.0, 0.1, 1.0)), ("pres", pick(0.0, 0.1, 1.5))):
        s[name] = torch.tensor(v, dtype=torch.float32).to(DEV)
    n_bias = [rng.randint(0, case["bias"]) for _ in range(R)]
    s["bias_start"] = ints([sum(n_bias[:r]) for r in range(R + 1)])
    s["bias_id"] = ints([v for n in n_bias for v in rng.sample(range(V), n)])
    s["bias_val"] = torch.tensor([rng.uniform(-5, 5) for _ in range(sum(n_bias))], dtype=torch.float32).to(DEV)
    # half of the requests answer within a grammar: every row has its own allowed set, of few tokens or of most
    rows = s["new"].tolist()
    kind = [rng.choice([0, 0, 1, 2]) for _ in range(R)]
    which, keep = [], []
    for r in range(R):
        for _ in range(rows[r]):
            which.append(len(keep) if kind[r] else -1)
            keep += [0.01 if kind[r] == 1 else 0.97] if kind[r] else []
    s["allow_row"] = ints(which)
    words = (V + 31) // 32
    if keep:
        allowed = torch.rand((len(keep), words * 32), generator=gen, device=DEV) < torch.tensor(keep).to(DEV)[:, None]
        bit = torch.ones(32, dtype=torch.int64, device=DEV) << torch.arange(32, device=DEV)
        s["allow"] = (allowed.view(len(keep), words, 32) * bit).sum(-1).to(torch.uint32).view(torch.int32)
    else:
        s["allow"] = torch.zeros((1, words), dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------------ the pass
def run(s):
    if own:
        return run_own(s)
    return {"map": plain_map, "store": plain_store, "attn": plain_attention, "rules": plain_rules}[s["op"]](s)


def run_own(s):
    import speculative_decoding_drafter_markov_gb300 as dsp
    if s["op"] == "map":
        out = dsp.page_map(s["lens"], s["new"], s["table"], s["held"], s["free"], s["n_free"], page=s["page"], N=s["cap"],
                           parents=s["parents"], max_rows=s["max_rows"], err=s["err"])
        return dict(out, table=s["table"], free=s["free"])
    if s["op"] == "store":
        dsp.cache_store(s["k"], s["v"], s["slot"], s["k_cache"], s["v_cache"], err=s["err"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["op"] == "attn":
        return dsp.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["row_start"], mask=s["mask"],
                                  scale=s["scale"], max_rows=s["max_rows"], err=s["err"])
    return dsp.logit_rules(s["T"], s["row_start"], tok=s["tok"], mask=s["mask"], hist=s["hist"], hist_len=s["hist_len"],
                           prompt_len=s["prompt_len"], rep=s["rep"], freq=s["freq"], pres=s["pres"], bias_start=s["bias_start"],
                           bias_id=s["bias_id"], bias_val=s["bias_val"], allow=s["allow"], allow_row=s["allow_row"], err=s["err"])


def rows_of(s):
    """Request and place within it of every row."""
    i = torch.arange(s["N"], device=DEV)
    req = torch.bucketize(i, s["row_start"][1:].long(), right=True)
    return req, i - s["row_start"].long()[req]


def plain_map(s):
    P, table, free = s["page"], s["table"], s["free"]
    lens, new, held = s["lens"].long(), s["new"].long(), s["held"].long()
    need = (lens + new + P - 1) // P
    less, more = (held - need).clamp(min=0), (need - held).clamp(min=0)
    page = torch.arange(table.shape[1], device=DEV)[None, :]
    before = s["n_free"].long()
    # pages given back go on the stack so that the first is on top; pages taken come from the top
    back = (page >= need[:, None]) & (page < held[:, None])
    rank = (torch.cumsum(less, 0) - less)[:, None] + page - need[:, None]
    after = before + less.sum()
    spare = torch.full((1,), free.shape[0], device=DEV, dtype=torch.int64)
    longer = torch.cat([free, free[:1]])
    longer.scatter_(0, torch.where(back, after - 1 - rank, spare).view(-1), table.view(-1))
    free.copy_(longer[:-1])
    take = (page >= held[:, None]) & (page < need[:, None])
    rank = (torch.cumsum(more, 0) - more)[:, None] + page - held[:, None]
    at = (after - 1 - rank).clamp(0, free.shape[0] - 1)
    table.copy_(torch.where(take, free[at], table))
    row_start = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    i = torch.arange(s["cap"], device=DEV)
    req = torch.bucketize(i, row_start[1:], right=True)
    live = req < s["R"]
    req = req.clamp(max=s["R"] - 1)
    j = i - row_start[req]
    place = lens[req] + j
    slot = torch.where(live, table.long()[req, (place // P).clamp(max=table.shape[1] - 1)] * P + place % P, -1)
    out = {"held": need.int(), "n_free": (after - more.sum()).int(), "row_start": row_start.int(), "slot": slot.int()}
    if s["parents"] is None:
        out["pos"] = torch.where(live, place, 0).int()
    else:
        # ancestors: the closure of "is the parent of", (1 - A)^-1 for the parents' matrix A, row by row 0 or 1
        n = s["max_rows"]
        line = torch.zeros((s["R"] * n * n + 1), device=DEV)
        p = torch.cat([s["parents"].long(), torch.full((s["cap"] - s["N"],), -1, device=DEV)])
        line.scatter_(0, torch.where(live & (p >= 0), (req * n + j) * n + p, s["R"] * n * n), 1.0)
        A = line[:-1].view(s["R"], n, n)
        eye = torch.eye(n, device=DEV).expand_as(A)
        seen = torch.linalg.solve_triangular(eye - A, eye, upper=False, unitriangular=True).round().long()
        bits = torch.nn.functional.pad(seen, (0, s["W"] * 64 - n)).view(s["R"], n, s["W"], 64)
        words = (bits << torch.arange(64, device=DEV)).sum(-1)
        at = (req, j.clamp(max=n - 1))
        out["pos"] = torch.where(live, lens[req] + seen.sum(-1)[at] - 1, 0).int()
        out["mask"] = torch.where(live[:, None], words[at], 0)
    return dict(out, table=table, free=free)


def plain_store(s):
    page, off = s["slot"].long() // s["page"], s["slot"].long() % s["page"]
    s["k_cache"][page, :, off] = s["k"]
    s["v_cache"][page, :, off] = s["v"]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def visible(s, req, j, n):
    """[N, n] truth values: row i may see row j of its request."""
    to = torch.arange(n, device=DEV)
    if s["mask"] is None:
        return to[None, :] <= j[:, None]
    return ((s["mask"][:, to // 64] >> (to % 64)) & 1).bool()


def plain_attention(s):
    R, n, P = s["R"], s["max_rows"], s["page"]
    H, D, G = s["k_cache"].shape[1], s["k_cache"].shape[3], s["q"].shape[1] // s["k_cache"].shape[1]
    req, j = rows_of(s)
    lens, new = s["lens"].long(), s["new"].long()
    used = s["table"].clamp(min=0).long()
    width = used.shape[1] * P
    # keys and values of every request side by side: [R, H, tokens, D]
    k = s["k_cache"][used].float().transpose(1, 2).reshape(R, H, width, D)
    v = s["v_cache"][used].float().transpose(1, 2).reshape(R, H, width, D)
    q = torch.zeros((R, n, H * G, D), device=DEV)
    q[req, j] = s["q"].float()
    q = q.view(R, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(R, H, n * G, D)
    score = (q @ k.transpose(2, 3)).view(R, H, n, G, width) * s["scale"]
    token = torch.arange(width, device=DEV)
    inner = torch.zeros((R, n, n), dtype=torch.bool, device=DEV)
    inner[req, j] = visible(s, req, j, n) & (torch.arange(n, device=DEV)[None, :] < new[req][:, None])
    rel = token[None, :] - lens[:, None]
    see = (rel < 0)[:, None, :] | ((rel >= 0) & (rel < n))[:, None, :] & torch.gather(inner, 2, rel.clamp(0, n - 1)[:, None, :].expand(R, n, width))
    score = score.masked_fill(~see[:, None, :, None, :], -INF)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -INF, torch.zeros_like(top), top)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    # what no row of the request may see takes no part, whatever its bits are
    v = v.masked_fill((rel >= new[:, None])[:, None, :, None], 0.0)
    out = (e.view(R, H, n * G, width) @ v).view(R, H, n, G, D) / total.clamp(min=1e-37)
    lse = (top + torch.log(total)).squeeze(-1)
    pick = lambda x: x.permute(0, 2, 1, 3, *range(4, x.dim())).flatten(2, 3)[req, j]  # noqa: E731
    return {"out": pick(out).to(s["q"].dtype), "lse": pick(lse)}


def plain_rules(s):
    T, R, N, V = s["T"], s["R"], s["N"], s["T"].shape[1]
    req, j = rows_of(s)
    n = s["max_rows"]
    at = torch.arange(s["hist"].shape[1], device=DEV)[None, :]
    in_text, in_prompt = at < s["hist_len"][:, None], at < s["prompt_len"][:, None]
    token = s["hist"].long()
    prompt = torch.zeros((R, V), device=DEV).scatter_add_(1, token, (in_text & in_prompt).float())
    count = torch.zeros((R, V), device=DEV).scatter_add_(1, token, (in_text & ~in_prompt).float())
    # the rows a row continues, itself among them; the request's first row is the last token of its text
    to = torch.arange(n, device=DEV)
    path = visible(s, req, j, n) & (to >= 1)[None, :] & (to[None, :] < s["new"].long()[req][:, None])
    drafted = s["tok"].long()[(s["row_start"].long()[req][:, None] + to[None, :]).clamp(max=N - 1)]
    c = count[req].scatter_add_(1, drafted, path.float())
    said = (c > 0) | (prompt[req] > 0)
    z = T.float()
    rep, freq, pres = (s[k][req][:, None] for k in ("rep", "freq", "pres"))
    z = torch.where(said, torch.where(z > 0, z / rep, z * rep), z) - freq * c - pres * (c > 0)
    of = torch.bucketize(torch.arange(s["bias_id"].shape[0], device=DEV), s["bias_start"][1:].long(), right=True)
    bias = torch.zeros((R, V), device=DEV)
    bias[of, s["bias_id"].long()] = s["bias_val"]
    z = z + bias[req]
    v = torch.arange(V, device=DEV)
    allowed = ((s["allow"][s["allow_row"].clamp(min=0).long()][:, v // 32] >> (v % 32).int()) & 1).bool()
    return z.masked_fill(~allowed & (s["allow_row"] >= 0)[:, None], -INF).to(T.dtype)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    lens, new = lens_of(case)
    R, N = len(new), sum(new)
    size = {"bf16": 2, "f32": 4}.get(case.get("dtype"), 0)
    if case["op"] == "map":
        P, W = case["page"], (max(new) + 63) // 64 if case["tree"] else 0
        row = 8 + (4 + 8 * W if W else 0)  # slot and position, parent and mask words
        entries = sum((a + b - 1) // P - a // P + 1 for a, b in zip(lens, new))  # table entries that hold the rows
        return {"bytes": N * row + 4 * entries + 20 * R, "flops": 0}
    if case["op"] == "store":
        return {"bytes": N * (4 * case["H"] * case["D"] * size + 4), "flops": 0}
    if case["op"] == "attn":
        H, Hq, D, P = case["H"], case["Hq"], case["D"], case["page"]
        tokens = sum(lens) + N
        words = 8 * ((max(new) + 63) // 64) if case["tree"] else 0
        pairs = sum(n * a + (n * (n + 1) // 2) for a, n in zip(lens, new))
        return {"bytes": 2 * tokens * H * D * size + N * (Hq * (2 * D * size + 4) + words) + 4 * (tokens // P) + 8 * R, "flops": 4 * pairs * Hq * D}
    return {"bytes": N * case["V"] * 2 * size + N * (case["V"] // 16) + 4 * sum(lens), "flops": 4 * N * case["V"]}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"map": exact_map, "store": exact_store, "attn": exact_attention, "rules": exact_rules}[case["op"]](s)


def exact_map(s):
    P, lens, new, held = s["page"], s["lens"].tolist(), s["new"].tolist(), s["held"].tolist()
    table, free, n = s["table"].cpu().numpy(), s["free"].cpu().numpy(), int(s["n_free"])
    need = [-(-(a + b) // P) for a, b in zip(lens, new)]
    back = [table[r, i] for r in range(len(new)) for i in range(need[r], held[r])]
    for k, page in enumerate(reversed(back)):
        free[n + k] = page
    n += len(back)
    for r in range(len(new)):
        for i in range(held[r], need[r]):
            n -= 1
            table[r, i] = free[n]
    slot, pos, words, start = np.full(s["cap"], -1, np.int32), np.zeros(s["cap"], np.int32), None, [0]
    parents = s["parents"].tolist() if s["parents"] is not None else None
    if parents:
        words = np.zeros((s["cap"], s["W"]), np.uint64)
        words[:s["N"]] = mask_words(new, parents, s["W"])
    for r, (a, n_new) in enumerate(zip(lens, new)):
        depth = []
        for j in range(n_new):
            t = a + j
            slot[start[-1] + j] = table[r, t // P] * P + t % P
            p = parents[start[-1] + j] if parents else j - 1
            depth.append(depth[p] + 1 if p >= 0 else 0)
            pos[start[-1] + j] = a + depth[j]
        start.append(start[-1] + n_new)
    out = {"held": np.array(need, np.int32), "n_free": np.array([n], np.int32), "row_start": np.array(start, np.int32), "slot": slot, "pos": pos}
    if parents:
        out["mask"] = words.view(np.int64)
    return dict(out, table=table, free=free)


def exact_store(s):
    k, v = s["k_cache"].double(), s["v_cache"].double()
    for name, cache in (("k", k), ("v", v)):
        flat = cache.transpose(1, 2).reshape(-1, cache.shape[1], cache.shape[3])
        flat[s["slot"].long()] = s[name].double()
        cache.copy_(flat.view(cache.shape[0], cache.shape[2], cache.shape[1], cache.shape[3]).transpose(1, 2))
    return {"k_cache": k, "v_cache": v}


def exact_attention(s):
    N, Hq, D = s["q"].shape
    P, H = s["page"], s["k_cache"].shape[1]
    out, lse = torch.zeros((N, Hq, D), dtype=torch.float64, device=DEV), torch.zeros((N, Hq), dtype=torch.float64, device=DEV)
    start = s["row_start"].tolist()
    for r, n_ctx in enumerate(s["lens"].tolist()):
        a, b = start[r], start[r + 1]
        t = torch.arange(n_ctx + b - a, device=DEV)
        page = s["table"][r].long()[t // P]
        see = torch.ones((b - a, len(t)), dtype=torch.bool, device=DEV)
        for j in range(b - a):
            word = [int(w) for w in s["mask"][a + j]] if s["mask"] is not None else None
            see[j, n_ctx:] = torch.tensor([(word[u // 64] >> (u % 64)) & 1 if word else u <= j for u in range(b - a)], dtype=torch.bool).to(DEV)
        for h in range(H):
            k, v = s["k_cache"][page, h, t % P].double(), s["v_cache"][page, h, t % P].double()
            for g in range(h * (Hq // H), (h + 1) * (Hq // H)):
                x = (s["q"][a:b, g].double() @ k.T * s["scale"]).masked_fill(~see, -INF)
                lse[a:b, g] = torch.logsumexp(x, 1)
                out[a:b, g] = torch.softmax(x, 1) @ v
    return {"out": out, "lse": lse}


def exact_rules(s):
    N, V = s["T"].shape
    out = torch.empty((N, V), dtype=torch.float64, device=DEV)
    start, bias_start = s["row_start"].tolist(), s["bias_start"].tolist()
    for r in range(s["R"]):
        text, n = s["hist"][r, :int(s["hist_len"][r])].long(), int(s["prompt_len"][r])
        base = torch.bincount(text[n:], minlength=V)
        in_prompt = torch.bincount(text[:n], minlength=V) > 0
        rep, freq, pres = (float(s[k][r]) for k in ("rep", "freq", "pres"))
        lo, hi = bias_start[r], bias_start[r + 1]
        for i in range(start[r], start[r + 1]):
            j = i - start[r]
            ahead = [u for u in range(1, start[r + 1] - start[r])
                     if (u <= j if s["mask"] is None else (int(s["mask"][i, u // 64]) >> (u % 64)) & 1)]
            c = base + torch.bincount(s["tok"][[start[r] + u for u in ahead]].long(), minlength=V)
            z = s["T"][i].double()
            z = torch.where((c > 0) | in_prompt, torch.where(z > 0, z / rep, z * rep), z) - freq * c - pres * (c > 0).double()
            z[s["bias_id"][lo:hi].long()] += s["bias_val"][lo:hi].double()
            m = int(s["allow_row"][i])
            if m >= 0:
                bits = (s["allow"][m].long()[:, None] >> torch.arange(32, device=DEV)) & 1
                z = z.masked_fill(bits.reshape(-1)[:V] == 0, -INF)
            out[i] = z
    return out
