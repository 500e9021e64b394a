"""The operators around the projections of a decoder layer: rotation of queries and keys with
their norms into a paged cache, attention of drafted tokens over that cache, and the cache's
pages (copying, forking, compacting, freeing). Cases, plain forms in elementary torch operations,
the library's calls, and the definitions in 64 bits.

A case is one call as it occurs between the binary-basis products: queries and keys of a
projection step come as its fp32 outputs (or as 16-bit rows of a fused buffer), a batch of
sequences has its keys and values in pages, and each sequence has a tree of up to 64 tokens
whose keys and values stand behind its context.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda:0"
F16, BF16, E4M3, F32 = torch.float16, torch.bfloat16, torch.float8_e4m3fn, torch.float32
TYPES = {"f16": F16, "bf16": BF16, "e4m3": E4M3, "f32": F32}
SIZE = {"f16": 2, "bf16": 2, "e4m3": 1, "f32": 4}
HEADS_70B, HEADS_7B = (64, 8), (32, 32)   # 8192 = 64 x 128 queries over 1024 = 8 x 128 keys; 4096 = 32 x 128


def listed():
    return [
        # the newest token of one sequence, right after the 70B q, k and v products: latency
        dict(name="rope one token", op="rope", tokens=1, heads=64, kv=8, dim=128, src="f32", cache="f16", rot=128,
             pairs=False, norm=False, page=16, reach=4096),
        # eight trees of 16 drafted tokens, rows of a fused buffer, normed, half of a head rotated
        dict(name="rope drafted trees", op="rope", tokens=128, heads=32, kv=32, dim=128, src="bf16", cache="bf16",
             rot=64, pairs=True, norm=True, page=32, reach=32768),
        # a long prompt into an 8-bit cache at far positions
        dict(name="rope prompt 8-bit", op="rope", tokens=8191, heads=64, kv=8, dim=128, src="f16", cache="e4m3",
             rot=128, pairs=False, norm=True, page=64, reach=1000000),
        # one token of one young sequence: latency
        dict(name="attend one token", op="attend", seqs=1, heads=32, kv=32, dim=128, cache="f16", q="f16", page=16,
             low=37, high=37, draft_low=1, draft_high=1, lens=1),
        # a serving batch of single tokens, contexts of very different lengths
        dict(name="attend batch ragged", op="attend", seqs=64, heads=64, kv=8, dim=128, cache="bf16", q="bf16",
             page=64, low=1, high=8192, draft_low=1, draft_high=1, lens=2),
        # eight sequences with 16 drafted tokens each (the largest batch of the products is 16 rows)
        dict(name="attend trees of 16", op="attend", seqs=8, heads=64, kv=8, dim=128, cache="f16", q="f16", page=16,
             low=16384, high=32700, draft_low=16, draft_high=16, lens=3),
        # wide trees over an 8-bit cache
        dict(name="attend trees of 64 8-bit", op="attend", seqs=4, heads=64, kv=8, dim=128, cache="e4m3", q="bf16",
             page=128, low=30001, high=65003, draft_low=64, draft_high=64, lens=4),
        # small heads, ragged trees, some sequences with no tokens or no context
        dict(name="attend ragged trees d64", op="attend", seqs=24, heads=12, kv=4, dim=64, cache="bf16", q="bf16",
             page=32, low=0, high=1500, draft_low=0, draft_high=40, lens=5),
        # a few pages of two layers: latency
        dict(name="copy few pages", op="copy", layers=2, pages=40, copies=3, kv=8, dim=128, cache="f16", page=16),
        # pages of 80 layers, as when many sequences fork or move
        dict(name="copy many pages", op="copy", layers=80, pages=600, copies=200, kv=8, dim=128, cache="bf16", page=16),
        # accepted tokens of 16 sequences drawn together behind their contexts, in 80 layers
        dict(name="compact accepted", op="compact", layers=80, seqs=16, kv=8, dim=128, cache="f16", page=16,
             low=100, high=900, draft=64, most=9, lens=6),
        # forks of running sequences with room reserved (their last page copied), older forks dropped
        dict(name="fork reserve free", op="fork", layers=4, seqs=256, parents=64, kv=8, dim=128, cache="f16", page=16,
             low=1, high=2000, room=64, lens=7),
    ]


def spread(rng, low, high):
    """A whole number in [low, high], spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.999)))))))


def draw(rng):
    op = rng.choice(["rope", "attend", "attend", "copy", "compact", "fork"])
    heads, kv = rng.choice([HEADS_70B, HEADS_7B, (12, 4), (16, 1), (40, 8), (5, 5)])
    dim = rng.choice([64, 128, 128, 256]) if heads * kv <= 512 else 128
    page = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["f16", "bf16", "e4m3"])
    half = rng.choice(["f16", "bf16"]) if cache == "e4m3" else cache
    if op == "rope":
        return dict(op=op, tokens=spread(rng, 1, 8000), heads=heads, kv=kv, dim=dim if heads * dim <= 8192 else 64,
                    src=rng.choice(["f32", half]), cache=cache, rot=rng.choice([dim // 4, dim // 2, dim]),
                    pairs=rng.random() < 0.5, norm=rng.random() < 0.5, page=page,
                    reach=spread(rng, 100, 1000000)) | (dict(dim=64, rot=32) if heads * dim > 8192 else {})
    if op == "attend":
        most = spread(rng, 1, 64)
        seqs = spread(rng, 1, 64)
        # no more than the largest listed case: rows x positions, and cache values
        high = spread(rng, 1, 65000)
        high = max(1, min(high, 4 * 64 * 64 * 47000 // (seqs * most * heads), 300000000 // (seqs * kv * dim)))
        return dict(op=op, seqs=seqs, heads=heads, kv=kv, dim=dim, cache=cache, q=half, page=page,
                    low=rng.choice([0, high // 2, high]), high=high, draft_low=rng.choice([0, 1, most]) if seqs > 1 else most,
                    draft_high=most, lens=rng.randrange(1 << 20))
    if op == "copy":
        layers = spread(rng, 1, 80)
        copies = spread(rng, 1, max(1, min(200, 16000 // layers * 16 * 1024 // (page * kv * dim))))
        return dict(op=op, layers=layers, pages=2 * copies + rng.randrange(1, 30), copies=copies, kv=kv, dim=dim,
                    cache=cache, page=page)
    if op == "compact":
        seqs, draft = spread(rng, 1, 24), spread(rng, 1, 64)
        return dict(op=op, layers=spread(rng, 1, 12), seqs=seqs, kv=kv, dim=dim, cache=cache, page=page, low=0,
                    high=spread(rng, 1, 300), draft=draft, most=spread(rng, 1, min(draft, 16)), lens=rng.randrange(1 << 20))
    seqs = spread(rng, 2, 300)
    return dict(op=op, layers=spread(rng, 1, 4), seqs=seqs, parents=max(1, seqs // rng.choice([2, 4, 7])), kv=kv, dim=64,
                cache=cache, page=page, low=0, high=spread(rng, 1, 2000), room=spread(rng, 1, 200),
                lens=rng.randrange(1 << 20))


# ----------------------------------------------------------------------------------------------
# sizes that belong to the case

def lengths(case):
    """Context lengths and tree sizes of an attention case (the first sequence has the longest)."""
    r = random.Random(case["lens"])
    ctx = [r.randint(case["low"], case["high"]) for _ in range(case["seqs"])]
    ctx[0] = case["high"]
    drafts = [r.randint(case["draft_low"], case["draft_high"]) for _ in range(case["seqs"])]
    drafts[0] = case["draft_high"]
    return ctx, drafts


def contexts(case):
    r = random.Random(case["lens"])
    return [r.randint(case["low"], case["high"]) for _ in range(case["seqs"])]


def kept(case):
    """For each sequence the drafted tokens that are accepted, ascending. Token i of a list is either
    in its place or comes from behind all places, so that a pass finds what the pass before it found."""
    r = random.Random(case["lens"] + 1)
    out = []
    for _ in range(case["seqs"]):
        m = r.randint(0, case["most"])
        free = [i for i in range(m, case["draft"])]
        stay = max(m - len(free), r.randint(0, m))
        out.append(list(range(stay)) + sorted(r.sample(free, m - stay)))
    return out


def forks(case):
    """Parent of each sequence (-1: none). The first `parents` sequences run, the others are forks."""
    r = random.Random(case["lens"] + 2)
    p = case["parents"]
    return [-1] * p + [r.randint(-1, p - 1) for _ in range(case["seqs"] - p)]


def fork_lens(case):
    r = random.Random(case["lens"] + 3)
    return [r.randint(case["low"], case["high"]) for _ in range(case["parents"])] + [0] * (case["seqs"] - case["parents"])


def fork_pages(case):
    """Pages enough for the parents, the rooms, and a quarter more."""
    ps, lens = case["page"], fork_lens(case)
    need = sum(-(-n // ps) for n in lens) + case["seqs"] * (case["room"] // ps + 2)
    return need + need // 4 + 1


def cdiv(a, b):
    return -(-a // b)


def work(case):
    op, size = case["op"], SIZE[case["cache"]]
    if op == "rope":
        t, h, k, d = (case[n] for n in ("tokens", "heads", "kv", "dim"))
        q = 2 if case["src"] == "f32" else SIZE[case["src"]]
        return {"bytes": t * d * ((h + 2 * k) * SIZE[case["src"]] + h * q + 2 * k * size) + 8 * t,
                "flops": t * d * (h + k) * (7 if case["norm"] else 3)}
    if op == "attend":
        ctx, drafts = lengths(case)
        h, k, d = case["heads"], case["kv"], case["dim"]
        live = [(c, n) for c, n in zip(ctx, drafts) if n]
        return {"bytes": sum(2 * (c + n) * k * d * size + n * h * (4 * d + 4) for c, n in live) + 4 * len(ctx),
                "flops": sum(4 * n * h * d * (c + (n + 1) / 2) for c, n in live) + 1}
    row = 2 * case["layers"] * case["kv"] * case["dim"] * size   # one token's keys and values in all layers
    if op == "copy":
        return {"bytes": 2 * case["copies"] * case["page"] * row, "flops": 0}
    if op == "compact":
        moved = sum(sum(1 for i, j in enumerate(js) if i != j) for js in kept(case))
        return {"bytes": 2 * moved * row + 4 * sum(len(js) for js in kept(case)) + 16, "flops": 0}
    ps, lens, par = case["page"], fork_lens(case), forks(case)
    shared = sum(cdiv(lens[p], ps) for p in par if p >= 0)
    part = sum(1 for p in par if p >= 0 and lens[p] % ps)
    room = len([p for p in par if p >= 0]) * cdiv(case["room"], ps)
    return {"bytes": 16 * shared + 24 * room + 2 * part * ps * row + 32 * case["seqs"], "flops": 0}


# ----------------------------------------------------------------------------------------------
# what a user's program has in hand

def values(shape, kind, gen, scale=None):
    """Normal values in a type; in 8 bits, what they are divided by comes per head (dimension -3)."""
    x = torch.empty(shape, dtype=TYPES[kind] if kind != "e4m3" else F16, device=DEV)
    for part in x.view(-1).split(1 << 28):
        part.normal_(generator=gen)
    if kind != "e4m3":
        return x
    y = torch.empty(shape, dtype=E4M3, device=DEV)
    for a, b in zip(y.view(-1, *shape[-3:]).split(1 << 10), x.view(-1, *shape[-3:]).split(1 << 10)):
        a.copy_((b.float() / scale[:, None, None]).clamp(-448, 448))
    return y


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def scales(case, gen):
    """What a head's 8-bit keys or values are multiplied by."""
    if case["cache"] != "e4m3":
        return None
    return torch.rand(case["kv"], device=DEV, generator=gen) * 0.05 + 0.01


def tables(lens, page, pages, seed):
    """Pages in an order of their own: a row for each sequence, -1 where it holds none."""
    rng = np.random.default_rng(seed)
    order = rng.permutation(pages).astype(np.int32)
    width = max(1, max(cdiv(n, page) for n in lens))
    held = np.array([cdiv(n, page) for n in lens])
    t = np.full((len(lens), width), -1, np.int32)
    t[np.arange(width)[None, :] < held[:, None]] = order[: held.sum()]
    return torch.from_numpy(t).to(DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op, kv, dim, page = case["op"], case["kv"], case["dim"], case["page"]
    s = dict(case=case, op=op, page=page, ks=scales(case, gen), vs=scales(case, gen))
    if op == "rope":
        t, h = case["tokens"], case["heads"]
        rows = torch.empty((t, (h + 2 * kv) * dim), dtype=TYPES[case["src"]], device=DEV).normal_(generator=gen)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, dim)) for x in rows.split([h * dim, kv * dim, kv * dim], 1))
        pages = cdiv(t, page) + 2
        s["kc"] = torch.zeros((pages, kv, page, dim), dtype=TYPES[case["cache"]], device=DEV)
        s["vc"] = torch.zeros_like(s["kc"])
        s["positions"] = torch.randint(0, case["reach"], (t,), dtype=torch.int32, device=DEV, generator=gen)
        order = torch.randperm(pages, device=DEV, generator=gen)
        at = torch.arange(t, device=DEV)
        s["slots"] = (order[at // page] * page + at % page).to(torch.int32)
        s["freq"] = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])
        s["freq"] = s["freq"].to(F32)
        s["qw"], s["kw"] = (torch.rand(dim, device=DEV, generator=gen) + 0.5 if case["norm"] else None for _ in "qk")
        s["half"] = case["src"] != "f32" and TYPES[case["src"]] or (F16 if case["cache"] == "e4m3" else TYPES[case["cache"]])
        s["out"] = torch.empty((t, h, dim), dtype=s["half"], device=DEV)
    elif op == "attend":
        ctx, drafts = lengths(case)
        full = [c + n for c, n in zip(ctx, drafts)]
        pages = sum(cdiv(n, page) for n in full) + 1
        s["kc"], s["vc"] = (values((pages, kv, page, dim), case["cache"], gen, x) for x in (s["ks"], s["vs"]))
        s["table"] = tables(full, page, pages, seed)
        s["ctx"], s["start"] = ints(ctx), ints([0] + list(np.cumsum(drafts)))
        s["longest"], s["widest"], t = max(full), max(drafts), sum(drafts)
        s["q"] = values((t, case["heads"], dim), case["q"], gen)
        r, masks = random.Random(seed), []
        for n in drafts:   # the token before it in the tree, drawn for each: it sees that one, what that one sees, and itself
            tree = []
            for i in range(n):
                tree.append((1 << i) | (tree[r.randint(max(0, i - 6), i - 1)] if i else 0))
            masks += [0 if n > 1 and r.random() < 1 / 16 else m for m in tree]   # some see the context alone
        s["masks"] = torch.from_numpy(np.array(masks, np.uint64).view(np.int64)).to(DEV)
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((t, case["heads"]), dtype=F32, device=DEV)
        if own:
            import ultra_bit_weight_uint32_amd as ubw
            s["cache"] = ubw.KVCache(s["kc"], s["vc"], k_scale=s["ks"], v_scale=s["vs"])
            s["plan"] = ubw.tree_attn_workspace(case["seqs"], s["widest"], case["heads"], kv, dim, device=DEV)
    else:
        layers = case["layers"]
        pages = case["pages"] if op == "copy" else fork_pages(case) if op == "fork" else None
        if op == "compact":
            full = [c + case["draft"] for c in contexts(case)]
            pages = sum(cdiv(n, page) for n in full) + 1
        shape = (layers, pages, kv, page, dim)
        s["kc"], s["vc"] = (values(shape, case["cache"], gen, x) for x in (s["ks"], s["vs"]))
        if op == "copy":
            order = torch.randperm(pages, device=DEV, generator=gen)[: 2 * case["copies"]]
            s["pairs"] = order.to(torch.int32).view(-1, 2)
        elif op == "compact":
            s["table"], s["ctx"] = tables(full, page, pages, seed), ints(contexts(case))
            js = kept(case)
            s["keep"] = ints([j + [-1] * (case["most"] - len(j)) for j in js]).view(case["seqs"], case["most"])
        else:
            lens = fork_lens(case)
            width = cdiv(case["high"] + case["room"], page) + 1
            t = tables(lens, page, pages, seed)
            s["table"] = torch.nn.functional.pad(t, (0, width - t.shape[1]), value=-1)
            s["len"], s["held"] = ints(lens), ints([cdiv(n, page) for n in lens])
            s["ref"] = torch.zeros(pages, dtype=torch.int32, device=DEV)
            s["ref"][t[t >= 0].long()] = 1
            s["free"] = free_words(s["ref"])
            s["status"] = ints([0])
            par = forks(case)
            s["parents"], s["drop"] = ints(par), ints([-1 if p < 0 else 0 for p in par])
            s["room"] = ints([0 if p < 0 else case["room"] for p in par])
            s["pairs"] = torch.full((case["seqs"], 2), -1, dtype=torch.int32, device=DEV)
            if own:
                import ultra_bit_weight_uint32_amd as ubw
                s["pool"] = ubw.PagePool(s["ref"], s["free"], s["table"], s["held"], s["len"], s["status"], page)
    if own and "cache" not in s:
        import ultra_bit_weight_uint32_amd as ubw
        s["cache"] = ubw.KVCache(s["kc"], s["vc"], k_scale=s["ks"], v_scale=s["vs"])
    return s


# ----------------------------------------------------------------------------------------------
# one pass

def seen(cache, scale):
    """A cache as the values it stands for."""
    if cache.dtype != E4M3:
        return cache
    return (cache.to(F32) * scale[:, None, None]).to(F16)


def raw(cache):
    """A cache's values by their bits: they are moved, not computed."""
    return cache.view(torch.int16 if cache.dtype != E4M3 else torch.uint8)


def free_words(ref):
    """Bit p % 32 of word p / 32: nothing holds page p."""
    bits = torch.nn.functional.pad((ref == 0).to(torch.int64), (0, -ref.numel() % 32)).view(-1, 32)
    words = (bits << torch.arange(32, device=ref.device)).sum(1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def run(s):
    if own:
        return run_own(s)
    return {"rope": plain_rope, "attend": plain_attend, "copy": plain_copy, "compact": plain_compact,
            "fork": plain_fork}[s["op"]](s)


def run_own(s):
    import ultra_bit_weight_uint32_amd as ubw
    op = s["op"]
    if op == "rope":
        ubw.qk_norm_rope(s["q"], s["k"], s["v"], s["cache"], s["positions"], s["slots"], s["freq"], q_weight=s["qw"],
                         k_weight=s["kw"], eps=1e-6, interleaved=s["case"]["pairs"], out=s["out"])
        return s["out"], seen(s["kc"], s["ks"]), seen(s["vc"], s["vs"])
    if op == "attend":
        ubw.tree_attn(s["q"], s["cache"], s["table"], s["start"], s["ctx"], s["masks"], max_tree=s["widest"],
                      max_len=s["longest"], out=s["out"], lse=s["lse"], workspace=s["plan"])
        return s["out"], s["lse"]
    if op == "copy":
        ubw.cache_copy_pages(s["cache"], s["pairs"])
    elif op == "compact":
        ubw.cache_compact(s["cache"], s["table"], s["ctx"], s["keep"])
    else:
        ubw.pages_trim(s["pool"], s["drop"])
        ubw.pages_fork(s["pool"], s["parents"])
        ubw.pages_reserve(s["pool"], s["room"], s["pairs"])
        ubw.cache_copy_pages(s["cache"], s["pairs"])
        return (raw(s["kc"]), raw(s["vc"]), s["pairs"], s["table"], s["ref"], s["free"], s["held"], s["len"], s["status"])
    return raw(s["kc"]), raw(s["vc"])


def plain_store(cache, scale, slots, x, page):
    """Rows x [T, heads, D] (32 bits) at the slots of a cache, in its type."""
    if cache.dtype == E4M3:
        x = (x / scale[:, None]).clamp(-448, 448)
    slots = slots.long()
    cache[slots // page, :, slots % page] = x.to(cache.dtype)


def plain_norm(x, w, eps):
    x = x.to(F32)
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w


def plain_rope(s):
    case = s["case"]
    rot, pairs = case["rot"], case["pairs"]
    angle = s["positions"].double()[:, None, None] * s["freq"].double()
    cos, sin = torch.cos(angle).to(F32), torch.sin(angle).to(F32)

    def turned(x):
        r, rest = x[..., :rot], x[..., rot:]
        if pairs:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = r[..., : rot // 2], r[..., rot // 2:]
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((r, rest), -1)

    s["out"].copy_(turned(plain_norm(s["q"], s["qw"], 1e-6)))
    plain_store(s["kc"], s["ks"], s["slots"], turned(plain_norm(s["k"], s["kw"], 1e-6)), s["page"])
    plain_store(s["vc"], s["vs"], s["slots"], s["v"].to(F32), s["page"])
    return s["out"], seen(s["kc"], s["ks"]), seen(s["vc"], s["vs"])


def plain_attend(s):
    ctx, start, page = s["ctx"].long(), s["start"].long(), s["page"]
    heads, kv, dim = s["q"].shape[1], s["kc"].shape[1], s["kc"].shape[3]
    seqs, wide = ctx.numel(), s["widest"]
    at = torch.arange(s["longest"], device=DEV)
    where = s["table"].long().clamp(min=0)[:, at // page]
    k = s["kc"][where, :, at % page].to(F32)                 # [seqs, positions, kv, D]
    v = s["vc"][where, :, at % page].to(F32)
    if s["ks"] is not None:
        k, v = k * s["ks"][:, None], v * s["vs"][:, None]
    counts = start[1:] - start[:-1]
    i = torch.arange(wide, device=DEV)
    row = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].to(F32) / math.sqrt(dim)                 # [seqs, wide, heads, D]
    q = q.view(seqs, wide, kv, heads // kv, dim).permute(0, 2, 3, 1, 4).reshape(seqs, kv, -1, dim)
    score = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()).view(seqs, kv, heads // kv, wide, -1)
    j = at - ctx[:, None]                                    # place in the tree, negative in the context
    bit = (s["masks"][row][:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1
    sees = (j[:, None, :] < 0) | ((bit == 1) & (j < counts[:, None])[:, None, :])
    score = score.masked_fill(~sees[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v.transpose(1, 2).contiguous()).view(seqs, kv, heads // kv, wide, dim)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(seqs, wide, heads, dim)
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(seqs, wide, heads)
    live = i < counts[:, None]
    s["out"].copy_(o[live])
    s["lse"].copy_(lse[live])
    return s["out"], s["lse"]


def plain_copy(s):
    a, b = s["pairs"][:, 0].long(), s["pairs"][:, 1].long()
    for c in (raw(s["kc"]), raw(s["vc"])):
        c[:, b] = c[:, a]
    return raw(s["kc"]), raw(s["vc"])


def plain_compact(s):
    ctx, keep, page = s["ctx"].long()[:, None], s["keep"].long(), s["page"]
    ok = keep >= 0
    src, dst = ctx + keep.clamp(min=0), ctx + torch.arange(keep.shape[1], device=DEV)
    table = s["table"].long()
    width = table.shape[1] - 1
    ps, pd = table.gather(1, (src // page).clamp(max=width))[ok], table.gather(1, (dst // page).clamp(max=width))[ok]
    src, dst = (src % page)[ok], (dst % page)[ok]
    for c in (raw(s["kc"]), raw(s["vc"])):
        c[:, pd, :, dst] = c[:, ps, :, src]
    return raw(s["kc"]), raw(s["vc"])


def plain_fork(s):
    page, table, held, length, ref = s["page"], s["table"], s["held"], s["len"], s["ref"]
    col = torch.arange(table.shape[1], device=DEV)
    # freeing: sequences cut to a length of drop (where it is not negative), pages behind it given back
    cut = torch.where(s["drop"] >= 0, (s["drop"] + page - 1) // page, held)
    gone = (col >= cut[:, None]) & (col < held[:, None])
    ref.index_add_(0, table[gone].long(), torch.full_like(table[gone], -1))
    table.masked_fill_(gone, -1)
    held.copy_(torch.minimum(held, cut))
    length.copy_(torch.where(s["drop"] >= 0, s["drop"], length))
    # forking: the parent's pages, shared
    par = s["parents"].long()
    child, n = par >= 0, length[par.clamp(min=0)]
    share = child[:, None] & (col < ((n + page - 1) // page)[:, None])
    table.copy_(torch.where(share, table[par.clamp(min=0)], table))
    ref.index_add_(0, table[share].long(), torch.ones_like(table[share]))
    held.copy_(torch.where(child, (n + page - 1) // page, held))
    length.copy_(torch.where(child, n, length))
    # room: pages for it, and one more where the last page is shared and has room left
    room, s["pairs"][:] = s["room"], -1
    last = table.gather(1, (length // page).long().clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    part = (room > 0) & (length // page < held) & (ref[last.long().clamp(min=0)] > 1)
    want = (torch.where(room > 0, (length + room + page - 1) // page, held) - held).clamp(min=0)
    need = want + part
    before = torch.cumsum(need, 0) - need
    free = torch.nonzero(ref == 0)[:, 0].to(torch.int32)
    s["pairs"][part] = torch.stack((last, free[before.clamp(max=free.numel() - 1)]), 1)[part]
    ref.index_add_(0, last[part].long(), torch.full_like(last[part], -1))
    at = torch.nonzero(part)[:, 0]
    table[at, (length // page).long()[at]] = s["pairs"][at, 1]
    new = (col >= held[:, None]) & (col < (held + want)[:, None])
    which = before[:, None] + part[:, None] + (col - held[:, None])
    table.copy_(torch.where(new, free[which.clamp(0, free.numel() - 1)], table))
    held.add_(want.to(torch.int32))
    taken = torch.cat((s["pairs"][part][:, 1], table[new])).long()
    ref.index_add_(0, taken, torch.ones(taken.numel(), dtype=torch.int32, device=DEV))
    s["free"].copy_(free_words(ref))
    a, b = s["pairs"][part][:, 0].long(), s["pairs"][part][:, 1].long()
    for c in (raw(s["kc"]), raw(s["vc"])):
        c[:, b] = c[:, a]
    return (raw(s["kc"]), raw(s["vc"]), s["pairs"], table, ref, s["free"], held, length, s["status"])


# ----------------------------------------------------------------------------------------------
# the definitions, in 64 bits

def to_e4m3(x):
    """The nearest value with 4 significant bits, exponents from -6 (below: steps of 2^-9), at most
    448; ties to the even one. x in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return exact_rope(s)
    if case["op"] == "attend":
        return exact_attend(s)
    return None


def exact_rope(s):
    case, rot = s["case"], s["case"]["rot"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       torch.outer(s["positions"].double(), s["freq"].double()))[:, None]

    def rotated(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * w.double()
        y = x.clone()
        if case["pairs"]:
            y[..., :rot] = torch.view_as_real(torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], -1, 2)) * turn).flatten(-2)
        else:
            z = torch.complex(x[..., : rot // 2], x[..., rot // 2:rot]) * turn
            y[..., :rot] = torch.cat((z.real, z.imag), -1)
        return y

    out = [rotated(s["q"], s["qw"])]
    for x, scale in ((rotated(s["k"], s["kw"]), s["ks"]), (s["v"].double(), s["vs"])):
        if scale is not None:
            x = to_e4m3(x / scale.double()[:, None]) * scale.double()[:, None]
        pages, _, page, _ = s["kc"].shape
        slots = torch.zeros((pages * page, *x.shape[1:]), dtype=torch.float64, device=DEV)
        slots[s["slots"].long()] = x
        out.append(slots.view(pages, page, *x.shape[1:]).transpose(1, 2).contiguous())
    return tuple(out)


def exact_attend(s):
    q, page = s["q"], s["page"]
    heads, kv, dim = q.shape[1], s["kc"].shape[1], q.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    start, ctx, masks = s["start"].tolist(), s["ctx"].tolist(), s["masks"].tolist()
    for b, c in enumerate(ctx):
        n = start[b + 1] - start[b]
        if not n:
            continue
        pages = s["table"][b, : cdiv(c + n, page)].long()
        rows = slice(start[b], start[b + 1])
        sees = torch.tensor([[True] * c + [bool(masks[t] >> j & 1) for j in range(n)] for t in range(rows.start, rows.stop)],
                            device=DEV) if c < 4096 else None
        if sees is None:
            tree = torch.tensor([[bool(masks[t] >> j & 1) for j in range(n)] for t in range(rows.start, rows.stop)], device=DEV)
            sees = torch.cat((torch.ones((n, c), dtype=torch.bool, device=DEV), tree), 1)
        for h in range(kv):
            k, v = (x[pages, h].reshape(-1, dim)[: c + n].double() for x in (s["kc"], s["vc"]))
            if s["ks"] is not None:
                k, v = k * s["ks"][h].double(), v * s["vs"][h].double()
            hs = slice(h * heads // kv, (h + 1) * heads // kv)
            x = torch.matmul(q[rows, hs].double().reshape(-1, dim), k.T.contiguous()).view(n, -1, c + n) / dim ** 0.5
            x[~sees[:, None].expand_as(x)] = -math.inf
            w = torch.nan_to_num(torch.softmax(x, -1))
            out[rows, hs] = torch.matmul(w.view(-1, c + n), v).view(n, -1, dim)
            lse[rows, hs] = torch.logsumexp(x, -1)
    return out, lse
