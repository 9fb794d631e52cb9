"""Cases of the operators on both sides of the paged key-value cache: the rotation of
queries and keys with their norms on the way into the cache, and a cache held in 4 bits
with the attention that reads it.

In the target's pass every layer, between its projection and its attention,

* norms the queries and keys of each head, rotates them by their positions and appends
  keys and values to the cache (``rope_store``),
* where the cache is held in 4 bits, writes keys and values as codes of 4 bits with a
  scale per 16 of them (``cache_store4``), and
* lets every row attend to that cache and to its own ancestors among the rows of the
  cycle (``tree_attention4``).

The cache in 4 bits: 16 neighbouring elements of a head share a scale s, one byte b:
s = 2^(b // 8 - 16) (1 + b % 8 / 8), b <= 254 (255: the 16 are not numbers).  An element
is n s with a whole number n of -7 .. 7, held as n + 8.  A page of a head is one run of
bytes, first the codes of its tokens (D / 2 bytes each), then their scales (D / 16 bytes
each); in the four bytes of eight elements, the low half of byte 0 is element 0, its high
half element 2, then 4 and 6, 1 and 3, 5 and 7.

``run`` computes a case in plain torch operations, or, with ``own`` set, by the
library's entry points.  ``exact`` computes it from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
INF = float("inf")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # plain decoding of a single request: one row, where latency counts
        dict(name="rope_single", op="rope", R=1, ctx=2047, rows=1, page=16, Hq=32, H=8, D=128, rot=128, pairs="halves", norm=True, cached=True, dtype="bf16"),
        # a cycle of 64 requests with chains of up to 9 rows behind texts of up to 32K tokens, one layer
        dict(name="rope_cycle", op="rope", R=64, ctx=32768, rows=9, page=16, Hq=32, H=8, D=128, rot=128, pairs="halves", norm=True, cached=True, dtype="bf16"),
        # a batch of prompts out of the fused query-key-value projection, one layer
        dict(name="rope_prompts", op="rope", R=24, ctx=0, rows=8192, page=64, Hq=32, H=8, D=128, rot=128, pairs="halves", norm=True, cached=True, dtype="bf16"),
        # in 32 bits, neighbouring elements rotated together, part of a head only, no norms; keys to a tensor of their own
        dict(name="rope_f32", op="rope", R=12, ctx=4000, rows=130, page=16, Hq=8, H=4, D=80, rot=40, pairs="neighbours", norm=False, cached=False, dtype="f32"),
        # one layer's write of a qwen4b cycle into a cache of 4 bits: 64 requests, up to 9 rows each
        dict(name="store4_cycle", op="store4", R=64, ctx=8192, rows=9, page=16, Hq=32, H=8, D=128, dtype="bf16"),
        # one layer's write of a batch of prompts
        dict(name="store4_prompts", op="store4", R=24, ctx=0, rows=8192, page=64, Hq=32, H=8, D=128, dtype="bf16"),
        # plain decoding of a single request
        dict(name="attn4_single", op="attn4", R=1, ctx=2047, rows=1, page=16, Hq=32, H=8, D=128, dtype="bf16", tree=False),
        # the tiny workload's precision: a few requests in 32 bits, chains of up to five rows
        dict(name="attn4_f32", op="attn4", R=4, ctx=1500, rows=5, page=16, Hq=8, H=4, D=64, dtype="f32", tree=False),
        # a qwen4b cycle: 64 requests with ragged caches and chains of up to 9 rows
        dict(name="attn4_chain", op="attn4", R=64, ctx=8192, rows=9, page=16, Hq=32, H=8, D=128, dtype="bf16", tree=False),
        # plain decoding of many requests, one row each: what the smaller cache makes room for
        dict(name="attn4_decode", op="attn4", R=128, ctx=16384, rows=1, page=64, Hq=64, H=8, D=128, dtype="bf16", tree=False),
        # trees of up to 64 candidates over 16K-token caches
        dict(name="attn4_tree", op="attn4", R=16, ctx=16384, rows=64, page=32, Hq=32, H=8, D=128, dtype="bf16", tree=True),
        # few requests with very long caches, chains of up to 17 rows
        dict(name="attn4_long", op="attn4", R=8, ctx=131072, rows=17, page=64, Hq=32, H=8, D=128, dtype="bf16", tree=False),
    ]


def log_int(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "store4", "attn4", "attn4", "attn4"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    R, G, H, D = log_int(rng, 1, 128), rng.choice([1, 2, 3, 4, 7, 8]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 128, 80, 96])
    c = dict(op=op, R=R, page=rng.choice([8, 16, 16, 32, 48, 64, 128]), Hq=G * H, H=H, D=D, dtype=dtype)
    if op == "attn4":
        rows = log_int(rng, 1, 64 if R <= 32 else 17)
        # tokens of all caches together: half of attn4_long's at most, an eighth in 32 bits, and not more pairs of a row's
        # head and a token than there
        most = min(524288 if dtype == "bf16" else 131072, 150000000 // (rows * G * H)) // R
        return dict(c, ctx=log_int(rng, 1, max(1, min(131072, most))), rows=rows, tree=rng.random() < 0.4)
    # bytes of the rows: no more than those of the prompts above
    most = 65536 * 40 * 128 * 2 // ((G + 2) * H * D * (2 if dtype == "bf16" else 4) * R)
    c.update(rows=log_int(rng, 1, max(1, min(8192, most))))
    if op == "store4":
        return dict(c, ctx=log_int(rng, 1, 4096))
    return dict(c, ctx=log_int(rng, 1, min(131072, 524288 // R)), rot=rng.choice([D, D, D // 2]), pairs=rng.choice(["halves", "halves", "neighbours"]),
                norm=rng.random() < 0.7, cached=rng.random() < 0.7)


def lens_of(case):
    """Cache lengths before the cycle and new rows of every request: whole numbers that the case alone gives."""
    rng = random.Random(case["R"] * 7919 + case["ctx"] * 31 + case["rows"])
    R, ctx, rows = case["R"], case["ctx"], case["rows"]
    lens = [ctx] + [log_int(rng, max(1, ctx // 16), ctx) if ctx else 0 for _ in range(R - 1)]
    new = [rows] + [log_int(rng, 1, rows) if rows > 64 else rng.randint(1, rows) for _ in range(R - 1)]
    return lens, new


# ------------------------------------------------------------------ inputs
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
PLACES = (0, 2, 4, 6, 1, 3, 5, 7)  # the element that each half byte of a code word holds


def ints(v):
    return torch.tensor(v, dtype=torch.int32).to(DEV)


def tree_masks(new, rng):
    """[N, W] 64-bit words of random trees: bit j of a row is set where row j of its request is the row or one of its
    ancestors, the parent of each one of the eight rows before it."""
    W, words = (max(new) + 63) // 64, []
    for n in new:
        seen = []
        for j in range(n):
            up = seen[rng.randint(max(0, j - 8), j - 1)] if j else 0
            seen.append(up | (1 << j))
        words += [[(s >> (64 * w)) & 0xFFFFFFFFFFFFFFFF for w in range(W)] for s in seen]
    return torch.tensor([[w - (1 << 64) if w >> 63 else w for w in row] for row in words], dtype=torch.int64).to(DEV)


def quantise(x):
    """Scale bytes [.., D / 16] and whole numbers [.., D] of rows [.., D], in 64 bits."""
    g = x.double().unflatten(-1, (-1, 16))
    most = g.abs().amax(-1)
    fits = most < INF
    want = torch.where(fits, most / 7, 1.0).clamp(2.0 ** -16, 57344.0)
    e = torch.floor(torch.log2(want))
    e = torch.where(torch.exp2(e) > want, e - 1, torch.where(torch.exp2(e + 1) <= want, e + 1, e))
    byte = 8 * (e + 16) + torch.round(want / torch.exp2(e) * 8) - 8  # round: halves go to the even neighbour
    s = scale_of(byte)
    n = torch.where(fits[..., None], torch.round(g / s[..., None]).clamp(-7, 7), 0.0)
    return torch.where(fits, byte, 255.0).to(torch.uint8), n.to(torch.int8).flatten(-2)


def scale_of(byte):
    b = byte.double()
    return torch.where(b == 255, float("nan"), torch.exp2(torch.floor(b / 8) - 16) * (1 + (b % 8) / 8))


def pack(n):
    """Code bytes [.., D / 2] of whole numbers [.., D]."""
    c = (n.to(torch.int16) + 8).unflatten(-1, (-1, 8))[..., list(PLACES)]
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8).flatten(-2)


def unpack(codes):
    """Whole numbers [.., D] as floats of code bytes [.., D / 2]."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8
    return n.unflatten(-1, (-1, 8))[..., [PLACES.index(i) for i in range(8)]].flatten(-2)


def values(cache, P, D):
    """Values [.., P, D] in 32 bits (which hold them exactly) of pages [.., P D 9 / 16]."""
    codes, scales = cache[..., :P * D // 2].unflatten(-1, (P, D // 2)), cache[..., P * D // 2:].unflatten(-1, (P, D // 16))
    return (unpack(codes).unflatten(-1, (-1, 16)) * scale_of(scales).float()[..., None]).flatten(-2)


def random_cache4(n_pages, H, P, D, gen):
    out = torch.empty((n_pages, H, P * D * 9 // 16), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (H * P * D))
    for a in range(0, n_pages, step):
        x = torch.randn((min(step, n_pages - a), H, P, D), generator=gen, device=DEV, dtype=torch.bfloat16)
        byte, n = quantise(x)
        out[a:a + step, :, :P * D // 2] = pack(n).flatten(2)
        out[a:a + step, :, P * D // 2:] = byte.flatten(2)
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
    H, Hq, D, dt, P = case["H"], case["Hq"], case["D"], TYPES[case["dtype"]], case["page"]
    s = dict(op=case["op"], N=start[-1], R=len(new), max_rows=max(new), lens=ints(lens), new=ints(new), row_start=ints(start), page=P,
             H=H, D=D, dt=dt, err=torch.zeros(1, dtype=torch.int32, device=DEV), mask=None, scale=1.0 / math.sqrt(D))
    need = [(a + b + P - 1) // P for a, b in zip(lens, new)]
    total, width = sum(need), max(need) + 2
    n_pages = total + total // 8 + 1
    order = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    used = torch.arange(width, device=DEV)[None, :] < ints(need)[:, None]
    table = torch.full((len(new), width), -1, dtype=torch.int32, device=DEV)
    table[used] = order[:total]
    # queries, keys and values out of one projection
    heads = torch.randn((s["N"], Hq + 2 * H, D), generator=gen, device=DEV, dtype=torch.float32).to(dt)
    s.update(table=table, q=heads[:, :Hq], k=heads[:, Hq:Hq + H], v=heads[:, Hq + H:])
    req, at = rows_of(s)
    place = s["lens"].long()[req] + at
    s["slot"] = (table.long()[req, place // P] * P + place % P).to(torch.int32)
    if case["op"] == "rope":
        s["pos"], s["rot"], s["halves"], s["cached"] = place.to(torch.int32), case["rot"], case["pairs"] == "halves", case["cached"]
        i = torch.arange(case["rot"] // 2, dtype=torch.float64)
        s["freq"] = torch.pow(torch.tensor(1e6, dtype=torch.float64), -2 * i / case["rot"]).float().to(DEV)
        for name in ("q_weight", "k_weight"):
            s[name] = (1 + 0.2 * torch.randn(D, generator=gen, device=DEV)).to(dt) if case["norm"] else None
        if case["cached"]:
            for name in ("k_cache", "v_cache"):
                s[name] = torch.randn((n_pages, H, P, D), generator=gen, device=DEV, dtype=dt)
        return s
    for name in ("k_cache", "v_cache"):
        s[name] = random_cache4(n_pages, H, P, D, gen)
    if case.get("tree"):
        s["mask"] = tree_masks(new, rng)
    return s


EPS = 1e-6  # of the norms


# ------------------------------------------------------------------ the pass
def run(s):
    if own:
        return run_own(s)
    return {"rope": plain_rope, "store4": plain_store4, "attn4": plain_attention4}[s["op"]](s)


def run_own(s):
    import speculative_decoding_drafter_markov_gb300 as dsp
    if s["op"] == "rope":
        norm = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=not s["halves"], err=s["err"])
        if not s["cached"]:
            return dsp.rope_store(s["q"], s["k"], None, s["pos"], s["freq"], **norm)
        o = dsp.rope_store(s["q"], s["k"], s["v"], s["pos"], s["freq"], slot=s["slot"], k_cache=s["k_cache"], v_cache=s["v_cache"], **norm)
        return {"q": o["q"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["op"] == "store4":
        o = dsp.cache_store4(s["k"], s["v"], s["slot"], s["k_cache"], s["v_cache"], values=True, err=s["err"])
        return {"k": o["k"], "v": o["v"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return dsp.tree_attention4(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["row_start"], mask=s["mask"], scale=s["scale"],
                               max_rows=s["max_rows"], err=s["err"])


def rows_of(s):
    """Request and place within it of every row."""
    i = torch.arange(s["N"], device=DEV)
    req = torch.bucketize(i, s["row_start"][1:].long(), right=True)
    return req, i - s["row_start"].long()[req]


def plain_rope(s):
    angle = s["pos"].double()[:, None] * s["freq"].double()
    c, n, half = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None], s["rot"] // 2

    def turn(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
        a, b = (x[..., :half], x[..., half:2 * half]) if s["halves"] else (x[..., 0:2 * half:2], x[..., 1:2 * half:2])
        two = (a * c - b * n, b * c + a * n)
        return torch.cat([torch.cat(two, -1) if s["halves"] else torch.stack(two, -1).flatten(-2), x[..., 2 * half:]], -1).to(s["dt"])

    q, k = turn(s["q"], s["q_weight"]), turn(s["k"], s["k_weight"])
    if not s["cached"]:
        return {"q": q, "k": k}
    page, off = s["slot"].long() // s["page"], s["slot"].long() % s["page"]
    s["k_cache"][page, :, off] = k
    s["v_cache"][page, :, off] = s["v"]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def plain_store4(s):
    P, D, out = s["page"], s["D"], {}
    page, off = s["slot"].long() // P, s["slot"].long() % P
    for name in ("k", "v"):
        byte, n = quantise(s[name])
        cache = s[name + "_cache"]
        cache[..., :P * D // 2].unflatten(-1, (P, D // 2))[page, :, off] = pack(n)
        cache[..., P * D // 2:].unflatten(-1, (P, D // 16))[page, :, off] = byte
        out[name] = (n.double().unflatten(-1, (-1, 16)) * scale_of(byte)[..., None]).flatten(-2).to(s["dt"])
    return dict(out, k_cache=s["k_cache"], v_cache=s["v_cache"])


def visible(s, j, n):
    """[N, n] truth values: row i may see row j of its request."""
    to = torch.arange(n, device=DEV)
    if s["mask"] is None:
        return to[None, :] <= j[:, None]
    return ((s["mask"][:, to // 64] >> (to % 64)) & 1).bool()


def plain_attention4(s):
    R, n, P, H, D, dt = s["R"], s["max_rows"], s["page"], s["H"], s["D"], s["dt"]
    G = s["q"].shape[1] // H
    req, j = rows_of(s)
    lens, new = s["lens"].long(), s["new"].long()
    pages = s["table"].clamp(min=0).long()
    width = pages.shape[1] * P
    # keys and values of every request side by side: [R, H, tokens, D]
    k, v = (values(s[c][pages], P, D).transpose(1, 2).reshape(R, H, width, D) for c in ("k_cache", "v_cache"))
    q = torch.zeros((R, n, H * G, D), device=DEV)
    q[req, j] = s["q"].float()
    q = q.view(R, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(R, H, n * G, D)
    score = (q @ k.transpose(2, 3)).view(R, H, n, G, width) * s["scale"]
    token = torch.arange(width, device=DEV)
    inner = torch.zeros((R, n, n), dtype=torch.bool, device=DEV)
    inner[req, j] = visible(s, j, n) & (torch.arange(n, device=DEV)[None, :] < new[req][:, None])
    rel = token[None, :] - lens[:, None]
    see = (rel < 0)[:, None, :] | ((rel >= 0) & (rel < n))[:, None, :] & torch.gather(inner, 2, rel.clamp(0, n - 1)[:, None, :].expand(R, n, width))
    score = score.masked_fill(~see[:, None, :, None, :], -INF)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -INF, torch.zeros_like(top), top)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    # what no row of the request may see takes no part, whatever its bytes are
    v = v.masked_fill((rel >= new[:, None])[:, None, :, None], 0.0)
    out = (e.view(R, H, n * G, width) @ v).view(R, H, n, G, D) / total.clamp(min=1e-37)
    lse = (top + torch.log(total)).squeeze(-1)
    pick = lambda x: x.permute(0, 2, 1, 3, *range(4, x.dim())).flatten(2, 3)[req, j]  # noqa: E731
    return {"out": pick(out).to(dt), "lse": pick(lse)}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    lens, new = lens_of(case)
    R, N, H, Hq, D, P = len(new), sum(new), case["H"], case["Hq"], case["D"], case["page"]
    size = {"bf16": 2, "f32": 4}[case["dtype"]]
    if case["op"] == "rope":
        heads = Hq + (2 * H if case["cached"] else H)
        per = 2 * case["rot"] + case["rot"] + (4 * D if case["norm"] else 0)  # of a head: products and sums
        return {"bytes": N * (2 * heads * D * size + (8 if case["cached"] else 4)), "flops": N * (Hq + H) * per}
    if case["op"] == "store4":
        # read; codes and scales; the values that they stand for
        return {"bytes": N * (2 * H * (2 * D * size + D * 9 // 16) + 4), "flops": N * 2 * H * D * 3}
    tokens = sum(lens) + N
    words = 8 * ((max(new) + 63) // 64) if case["tree"] else 0
    pairs = sum(n * a + (n * (n + 1) // 2) for a, n in zip(lens, new))
    return {"bytes": 2 * tokens * H * D * 9 // 16 + N * (Hq * (2 * D * size + 4) + words) + 4 * (tokens // P) + 8 * R, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": exact_rope, "store4": exact_store4, "attn4": exact_attention4}[case["op"]](s)


def exact_rope(s):
    half = s["rot"] // 2
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), s["pos"].double()[:, None] * s["freq"].double())

    def one(x, weight, out):
        # head by head, as complex numbers
        for h in range(x.shape[1]):
            y = x[:, h].double()
            if weight is not None:
                y = y / (torch.linalg.vector_norm(y, dim=1, keepdim=True) ** 2 / s["D"] + EPS).sqrt() * weight.double()
            order = torch.arange(2 * half, device=DEV).view(2, half).T.reshape(-1) if s["halves"] else torch.arange(2 * half, device=DEV)
            z = torch.view_as_complex(y[:, order].reshape(-1, half, 2)) * turn
            y[:, order] = torch.view_as_real(z).reshape(-1, 2 * half)
            out(h, y)

    q = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    k = torch.empty(s["k"].shape, dtype=torch.float64, device=DEV)
    one(s["q"], s["q_weight"], lambda h, y: q[:, h].copy_(y))
    one(s["k"], s["k_weight"], lambda h, y: k[:, h].copy_(y))
    if not s["cached"]:
        return {"q": q, "k": k}
    res = {"q": q}
    for name, rows in (("k_cache", k), ("v_cache", s["v"].double())):
        flat = s[name].double().transpose(1, 2).reshape(-1, s["H"], s["D"])
        flat[s["slot"].long()] = rows
        res[name] = flat.view(-1, s["page"], s["H"], s["D"]).transpose(1, 2)
    return res


def exact_store4(s):
    P, D, H, N = s["page"], s["D"], s["H"], s["N"]
    res = {}
    # every scale there is, and halfway to the next: where a value is just there the even byte is taken
    every = scale_of(torch.arange(255, device=DEV))
    half = (every[1:] + every[:-1]) / 2
    for name in ("k", "v"):
        x = s[name].double().reshape(N, H, D // 16, 16)
        a = x.abs().amax(-1) / 7
        above, reached = torch.bucketize(a, half), torch.bucketize(a, half, right=True)
        byte = torch.where((above % 2 == 1) & (reached > above), reached, above)
        byte = torch.where(a < INF, byte, 255)
        step = every[byte.clamp(max=254)][..., None]
        low = torch.floor(x / step)
        over = x - (low + 0.5) * step  # (exact: few bits each)
        n = torch.where(over > 0, low + 1, torch.where(over < 0, low, low + torch.remainder(low, 2)))
        n = n.clamp(-7, 7)
        res[name] = (n * torch.where(byte < 255, every[byte.clamp(max=254)], float("nan"))[..., None]).reshape(N, H, D)
        code = torch.where(byte[..., None] < 255, n + 8, 8.0).long().reshape(N, H, D // 8, 8)
        by = torch.stack([code[..., 0] + 16 * code[..., 2], code[..., 4] + 16 * code[..., 6], code[..., 1] + 16 * code[..., 3],
                          code[..., 5] + 16 * code[..., 7]], -1).reshape(N, H, D // 2)
        cache = s[name + "_cache"]
        page, off = s["slot"].long() // P, s["slot"].long() % P
        for h in range(H):
            codes = cache[:, h, :P * D // 2].clone().view(-1, D // 2)
            codes[page * P + off] = by[:, h].to(torch.uint8)
            cache[:, h, :P * D // 2] = codes.view(-1, P * D // 2)
            scales = cache[:, h, P * D // 2:].clone().view(-1, D // 16)
            scales[page * P + off] = byte[:, h].to(torch.uint8)
            cache[:, h, P * D // 2:] = scales.view(-1, P * D // 16)
        res[name + "_cache"] = cache
    return res


def exact_attention4(s):
    N, Hq, D = s["q"].shape
    P, H = s["page"], s["H"]
    out, lse = torch.zeros((N, Hq, D), dtype=torch.float64, device=DEV), torch.zeros((N, Hq), dtype=torch.float64, device=DEV)
    start = s["row_start"].tolist()
    spread = torch.tensor([4 * i if i < 4 else 16 + 4 * (i - 4) for i in range(8)], device=DEV)  # bit of each half byte
    element = torch.tensor([(i % 2) * 4 + i // 2 for i in range(8)], device=DEV)  # half byte of each element

    def tokens(cache, r, n, h):
        t = torch.arange(n, device=DEV)
        page, off = s["table"][r].long()[t // P], t % P
        by = cache[:, h][page[:, None], off[:, None] * (D // 2) + torch.arange(D // 2, device=DEV)].long().view(n, D // 8, 4)
        word = by[..., 0] + (by[..., 1] << 8) + (by[..., 2] << 16) + (by[..., 3] << 24)
        code = ((word[..., None] >> spread[element]) & 15).double().view(n, D // 16, 16) - 8
        b = cache[:, h][page[:, None], P * D // 2 + off[:, None] * (D // 16) + torch.arange(D // 16, device=DEV)].long()
        s16 = torch.ldexp((8 + b % 8).double(), b // 8 - 19)
        return (code * s16[..., None]).view(n, D)

    for r, n_ctx in enumerate(s["lens"].tolist()):
        a, b = start[r], start[r + 1]
        see = torch.ones((b - a, n_ctx + b - a), dtype=torch.bool, device=DEV)
        for j in range(b - a):
            word = [int(w) for w in s["mask"][a + j]] if s["mask"] is not None else None
            see[j, n_ctx:] = torch.tensor([(word[u // 64] >> (u % 64)) & 1 if word else u <= j for u in range(b - a)], dtype=torch.bool).to(DEV)
        for h in range(H):
            k, v = tokens(s["k_cache"], r, n_ctx + b - a, h), tokens(s["v_cache"], r, n_ctx + b - a, h)
            for g in range(h * (Hq // H), (h + 1) * (Hq // H)):
                x = (s["q"][a:b, g].double() @ k.T * s["scale"]).masked_fill(~see, -INF)
                lse[a:b, g] = torch.logsumexp(x, 1)
                out[a:b, g] = torch.softmax(x, 1) @ v
    return {"out": out, "lse": lse}
