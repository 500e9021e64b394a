"""Attention over a paged key/value cache that need not read all of it for each sequence: a prefix that
several sequences share is gone through once for all of them, and a query attends to the blocks (pages)
of its context that a cheap score selects, with the bounds of each block's keys that the score is made of.
Cases, plain forms in elementary torch operations, the library's calls, and the definitions in 64 bits.

A case is one call of one layer's decoding step (or, for the bounds, of all layers once a step): a batch
of sequences, each with one new token or a tree of up to 64 drafted ones whose keys and values stand
behind its context.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda:0"
F16, BF16, E4M3, F32, F64 = torch.float16, torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.float64
TYPES = {"f16": F16, "bf16": BF16, "e4m3": E4M3}
SIZE = {"f16": 2, "bf16": 2, "e4m3": 1}
HEADS_70B, HEADS_7B = (64, 8), (32, 32)   # 8192 = 64 x 128 queries over 1024 = 8 x 128 keys; 4096 = 32 x 128


def listed():
    return [
        # four samples of one prompt, a few tokens in: latency
        dict(name="prefix four samples", op="prefix", seqs=4, groups=1, heads=64, kv=8, dim=128, cache="f16", q="f16",
             page=16, plow=1000, phigh=1000, low=1, high=40, draft_low=1, draft_high=1, lens=1),
        # 64 samples of one long prompt, each with an answer of its own by now
        dict(name="prefix 64 samples", op="prefix", seqs=64, groups=1, heads=64, kv=8, dim=128, cache="bf16", q="bf16",
             page=64, plow=16384, phigh=16384, low=1, high=2000, draft_low=1, draft_high=1, lens=2),
        # five system prompts, trees of drafted tokens, an 8-bit cache: the largest
        dict(name="prefix ragged trees 8-bit", op="prefix", seqs=32, groups=5, heads=64, kv=8, dim=128, cache="e4m3",
             q="bf16", page=128, plow=3001, phigh=40003, low=0, high=600, draft_low=1, draft_high=16, lens=3),
        # every query head with keys of its own, some sequences without tokens or without any of their own
        dict(name="prefix 32 heads", op="prefix", seqs=40, groups=3, heads=32, kv=32, dim=128, cache="f16", q="f16",
             page=32, plow=501, phigh=8191, low=0, high=300, draft_low=0, draft_high=3, lens=4),
        # the pages that a step of 64 sequences filled, in all layers: few or none
        dict(name="bounds decoding step", op="bounds", layers=80, seqs=64, kv=8, dim=128, cache="f16", page=16, low=100,
             high=700, most=16, lens=5),
        # a prompt just stored
        dict(name="bounds long prompt", op="bounds", layers=4, seqs=1, kv=8, dim=128, cache="bf16", page=32, low=0, high=0,
             most=50001, lens=6),
        # one token over a long context: latency
        dict(name="select one token", op="select", seqs=1, heads=64, kv=8, dim=128, cache="f16", q="f16", page=16,
             low=30011, high=30011, draft_low=1, draft_high=1, count=128, first=1, last=4, lens=7),
        # a serving batch of contexts of very different lengths
        dict(name="select ragged batch", op="select", seqs=64, heads=64, kv=8, dim=128, cache="bf16", q="bf16", page=32,
             low=1, high=65000, draft_low=1, draft_high=1, count=64, first=1, last=2, lens=8),
        # trees of 16 over far contexts in 8 bits
        dict(name="select trees of 16 8-bit", op="select", seqs=8, heads=64, kv=8, dim=128, cache="e4m3", q="bf16", page=32,
             low=40000, high=130000, draft_low=16, draft_high=16, count=96, first=2, last=3, lens=9),
        # one token, 2048 selected positions: latency
        dict(name="blocks one token", op="blocks", seqs=1, heads=64, kv=8, dim=128, cache="f16", q="f16", page=16,
             low=30011, high=30011, draft_low=1, draft_high=1, count=128, lens=10),
        # the serving batch
        dict(name="blocks ragged batch", op="blocks", seqs=64, heads=64, kv=8, dim=128, cache="bf16", q="bf16", page=32,
             low=1, high=16000, draft_low=1, draft_high=1, count=64, lens=11),
        # trees of 16, whose tokens share most of their blocks, in 8 bits
        dict(name="blocks trees of 16 8-bit", op="blocks", seqs=8, heads=64, kv=8, dim=128, cache="e4m3", q="bf16", page=64,
             low=20000, high=60000, draft_low=16, draft_high=16, count=64, lens=12),
    ]


def spread(rng, low, high):
    """A whole number in [low, high], spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.999)))))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "bounds", "select", "blocks", "blocks"])
    heads, kv = rng.choice([HEADS_70B, HEADS_7B, (12, 4), (16, 1), (40, 8), (5, 5)])
    dim = rng.choice([64, 128, 128, 256]) if heads * kv <= 512 else 128
    page = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["f16", "bf16", "e4m3"])
    half = rng.choice(["f16", "bf16"]) if cache == "e4m3" else cache
    lens = rng.randrange(1 << 20)
    base = dict(op=op, kv=kv, dim=dim, cache=cache, page=page, lens=lens)
    if op == "bounds":
        layers, seqs = spread(rng, 1, 80), spread(rng, 1, 64)
        most = spread(rng, page, max(page, min(50000, 4 * 50000 * 8 * 128 // (layers * seqs * kv * dim))))
        high = spread(rng, 1, max(1, min(2000, 200000000 // (layers * seqs * kv * dim))))
        return base | dict(layers=layers, seqs=seqs, low=rng.choice([0, high]), high=high, most=most)
    seqs, wide = spread(rng, 1, 64), rng.choice([1, 1, spread(rng, 1, 64)])
    low = rng.choice([0, 1, wide]) if seqs > 1 else wide
    base |= dict(seqs=seqs, heads=heads, q=half, draft_low=min(low, wide), draft_high=wide)
    if op == "prefix":
        # no more than the largest listed case: rows x positions, and cache values
        high = spread(rng, 1, max(1, min(2000, 60000000 // (seqs * kv * dim))))
        phigh = spread(rng, 1, max(1, min(40000, 25000000000 // (seqs * wide * heads * dim), 100000000 // (kv * dim))))
        groups = spread(rng, 1, max(1, min(seqs, 8, 120000000 // (phigh * kv * dim))))
        return base | dict(groups=groups, plow=rng.choice([0, phigh // 2, phigh]), phigh=phigh,
                           low=rng.choice([0, high // 2, high]), high=high)
    count = spread(rng, 1, 256)
    if op == "select":
        high = spread(rng, 40 * page, max(40 * page, min(130000, 400000000 * page // (seqs * kv * dim * 8),
                                                         1400000000 // (seqs * wide * kv * dim) * page)))
        count = min(count, high // page // 2)   # some are left out
        first = min(rng.choice([0, 1, 2]), count - 1)
        return base | dict(low=rng.choice([0, high // 2, high]), high=high, count=count, first=first,
                           last=min(rng.choice([0, 1, 4]), count - 1 - first))
    count = max(1, min(count, 64 * 64 * 128 * 8 * 16 // (seqs * wide * page * kv),
                       125000000 // (seqs * kv * dim * page * (8 + wide)) * 8))
    high = spread(rng, 1, max(1, min(60000, 500000000 // (seqs * kv * dim))))
    return base | dict(low=rng.choice([0, high // 2, high]), high=high, count=count)


# ----------------------------------------------------------------------------------------------
# sizes that belong to the case

def cdiv(a, b):
    return -(-a // b)


def lengths(case):
    """Context lengths and tree sizes (the first sequence has the longest)."""
    r = random.Random(case["lens"])
    ctx = [r.randint(case["low"], case["high"]) for _ in range(case["seqs"])]
    ctx[0] = case["high"]
    drafts = [r.randint(case["draft_low"], case["draft_high"]) for _ in range(case["seqs"])]
    drafts[0] = case["draft_high"]
    return ctx, drafts


def groups_of(case):
    """First sequence of each group (and the end), and the groups' prefix lengths."""
    r = random.Random(case["lens"] + 1)
    cuts = sorted(r.sample(range(1, case["seqs"]), case["groups"] - 1))
    prefix = [r.randint(case["plow"], case["phigh"]) for _ in range(case["groups"])]
    prefix[0] = case["phigh"]
    return [0] + cuts + [case["seqs"]], prefix


def steps(case):
    """Old and new length of each sequence."""
    r = random.Random(case["lens"])
    old = [r.randint(case["low"], case["high"]) for _ in range(case["seqs"])]
    new = [n + r.randint(1, case["most"]) for n in old]
    new[0] = old[0] + case["most"]
    return old, new


def lists(case):
    """For each sequence: whole blocks of its context, entries of a token's list, and those of them that
    the token shares with no other one."""
    out = []
    for c, n in zip(*lengths(case)):
        whole = c // case["page"]
        m = min(whole, case["count"])
        out.append((whole, m, min(m // 8, (whole - m) // (n - 1)) if n > 1 else 0))
    return out


def work(case):
    op, size, k, d = case["op"], SIZE[case["cache"]], case["kv"], case["dim"]
    page = case["page"]
    if op == "bounds":
        full = sum(new // page - old // page for old, new in zip(*steps(case)))
        return {"bytes": case["layers"] * full * k * d * size * (page + 2) + 8 * case["seqs"],
                "flops": 2 * case["layers"] * full * k * d * page}
    ctx, drafts = lengths(case)
    h = case["heads"]
    rows = sum(drafts) * h * (4 * d + 4)   # queries, outputs, log-sums
    if op == "prefix":
        start, prefix = groups_of(case)
        moved, pairs = 0, 0
        for g, p in enumerate(prefix):
            members = [(ctx[b], drafts[b]) for b in range(start[g], start[g + 1]) if drafts[b]]
            moved += (p if members else 0) + sum(c + n for c, n in members)
            pairs += sum(n * (p + c + (n + 1) / 2) for c, n in members)
        return {"bytes": 2 * moved * k * d * size + rows + 4 * len(ctx), "flops": 4 * pairs * h * d + 1}
    if op == "select":
        blocks = sum(c // page for c, n in zip(ctx, drafts) if n)
        each = sum(c // page * n for c, n in zip(ctx, drafts))
        return {"bytes": blocks * k * 2 * d * size + sum(drafts) * (h * d * 2 + k * case["count"] * 4) + 4 * blocks,
                "flops": 4 * each * k * d + 1}
    moved, pairs = 0, 0
    for (whole, m, fresh), c, n in zip(lists(case), ctx, drafts):
        if n:
            moved += (m - fresh + n * fresh) * page + c % page + n
            pairs += n * (m * page + c % page + (n + 1) / 2)
    return {"bytes": 2 * moved * k * d * size + rows + 4 * sum(drafts) * k * case["count"], "flops": 4 * pairs * h * d + 1}


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


def tree_masks(drafts, seed):
    """The token before each one in its tree is drawn; it sees that one, what that one sees, and itself."""
    r, masks = random.Random(seed), []
    for n in drafts:
        tree = []
        for i in range(n):
            tree.append((1 << i) | (tree[r.randint(max(0, i - 6), i - 1)] if i else 0))
        masks += [0 if n > 1 and r.random() < 1 / 16 else m for m in tree]   # some see the context alone
    return torch.from_numpy(np.array(masks, np.uint64).view(np.int64)).to(DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    op, kv, dim, page = case["op"], case["kv"], case["dim"], case["page"]
    s = dict(case=case, op=op, page=page, ks=scales(case, gen), vs=scales(case, gen))
    if op == "bounds":
        old, full = steps(case)
    else:
        ctx, drafts = lengths(case)
        t = sum(drafts)
        s["start"], s["widest"] = ints([0] + list(np.cumsum(drafts))), max(drafts)
        s["q"] = values((t, case["heads"], dim), case["q"], gen)
        s["masks"] = tree_masks(drafts, seed)
        if op == "prefix":
            first, prefix = groups_of(case)
            for g, p in enumerate(prefix):
                for b in range(first[g], first[g + 1]):
                    ctx[b] += p
        full = [c + n for c, n in zip(ctx, drafts)]
        s["ctx"], s["longest"], s["apart"] = ints(ctx), max(full), max(c + n for c, n in zip(*lengths(case)))

    # pages in an order of their own: a row for each sequence, -1 where it holds none
    held = np.array([cdiv(n, page) for n in full])
    table = np.full((len(full), max(1, held.max())), -1, np.int32)
    mine = np.arange(table.shape[1])[None, :] < held[:, None]
    copies = []
    if op == "prefix":   # samples hold the whole pages of their prefix together, and a copy each of its last one
        for g, p in enumerate(prefix):
            mine[first[g] + 1: first[g + 1], : p // page] = False
    pages = int(mine.sum()) + 1
    table[mine] = rng.permutation(pages).astype(np.int32)[: pages - 1]
    if op == "prefix":
        for g, p in enumerate(prefix):
            lead, rest = first[g], slice(first[g] + 1, first[g + 1])
            table[rest, : p // page] = table[lead, : p // page]
            if p % page:
                copies += [(table[lead, p // page], x) for x in table[rest, p // page]]
        s["first"], s["prefix"] = ints(first), ints(prefix)
    s["table"] = torch.from_numpy(table).to(DEV)

    if op == "select":   # bounds around a block's middle
        mid, half = (torch.empty((pages, kv, dim), device=DEV).normal_(generator=gen) for _ in "mh")
        b = torch.stack((mid - half.abs(), mid + half.abs()), 2)
        s["bounds"] = (b if s["ks"] is None else (b / s["ks"][:, None, None]).clamp(-448, 448)).to(TYPES[case["cache"]])
        s["out"] = torch.full((t, kv, case["count"]), -1, dtype=torch.int32, device=DEV)
    elif op == "bounds":
        shape = (case["layers"], pages, kv, page, dim)
        s["kc"] = values(shape, case["cache"], gen, s["ks"])
        s["bounds"] = torch.zeros((case["layers"], pages, kv, 2, dim), dtype=TYPES[case["cache"]], device=DEV)
        s["old"], s["new"], s["most"] = ints(old), ints(full), max(n - o for o, n in zip(old, full))
    else:
        s["kc"], s["vc"] = (values((pages, kv, page, dim), case["cache"], gen, x) for x in (s["ks"], s["vs"]))
        if copies:
            a, b = torch.tensor(np.array(copies).T.astype(np.int64), device=DEV)
            for c in (s["kc"], s["vc"]):
                raw = c.view(torch.uint8)
                raw[b] = raw[a]
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((t, case["heads"]), dtype=F32, device=DEV)
    if op == "blocks":   # a token's blocks: most are its sequence's, some its own
        sel = np.full((t, kv, case["count"]), -1, np.int32)
        row = 0
        for (whole, m, fresh), n in zip(lists(case), drafts):
            for h in range(kv):
                order = rng.permutation(whole).astype(np.int32)
                for i in range(n):
                    at = m - fresh + i * fresh
                    sel[row + i, h, :m] = np.sort(np.concatenate((order[: m - fresh], order[at: at + fresh])))
            row += n
        s["blocks"] = torch.from_numpy(sel).to(DEV)
    if own:
        import ultra_bit_weight_uint32_amd as ubw
        if op == "bounds":   # the call reads keys alone
            s["handle"] = ubw.KVCache(s["kc"], s["kc"], k_scale=s["ks"], v_scale=s["vs"])
        elif op == "select":
            s["plan"] = ubw.block_select_workspace(t, kv, table.shape[1], device=DEV)
        else:
            s["handle"] = ubw.KVCache(s["kc"], s["vc"], k_scale=s["ks"], v_scale=s["vs"])
            if op == "prefix":
                s["plan"] = ubw.prefix_attn_workspace(case["seqs"], case["groups"], t, s["widest"], case["heads"], kv, dim,
                                                      device=DEV)
            else:
                s["plan"] = ubw.block_attn_workspace(t, case["heads"], kv, dim, device=DEV)
    return s


# ----------------------------------------------------------------------------------------------
# one pass

def run(s):
    if own:
        return run_own(s)
    return {"prefix": plain_prefix, "bounds": plain_bounds, "select": plain_select, "blocks": plain_blocks}[s["op"]](s)


def whole_values(bounds):
    """Bounds as the values they stand for."""
    return bounds.to(F16) if bounds.dtype == E4M3 else bounds


def run_own(s):
    import ultra_bit_weight_uint32_amd as ubw
    case, op = s["case"], s["op"]
    if op == "prefix":
        ubw.prefix_attn(s["q"], s["handle"], s["table"], s["start"], s["ctx"], s["first"], s["prefix"], s["masks"],
                        max_tree=s["widest"], max_len=s["longest"], out=s["out"], lse=s["lse"], workspace=s["plan"])
        return s["out"], s["lse"]
    if op == "bounds":
        ubw.page_bounds(s["handle"], s["bounds"], s["table"], s["old"], s["new"], max_new=s["most"])
        return whole_values(s["bounds"])
    if op == "select":
        return ubw.block_select(s["q"], s["bounds"], s["table"], s["start"], s["ctx"], case["count"], page_size=s["page"],
                                first=case["first"], last=case["last"], max_tree=s["widest"], max_len=s["longest"],
                                out=s["out"], workspace=s["plan"])
    ubw.block_attn(s["q"], s["handle"], s["table"], s["start"], s["ctx"], s["blocks"], s["masks"], max_tree=s["widest"],
                   out=s["out"], lse=s["lse"], workspace=s["plan"])
    return s["out"], s["lse"]


def rows_of(s):
    """Rows of q by sequence and token (padded to the widest), and the tokens' number of each sequence."""
    start = s["start"].long()
    counts = start[1:] - start[:-1]
    i = torch.arange(s["widest"], device=DEV)
    return (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1), counts, i < counts[:, None]


def gathered(s, where, at):
    """Keys and values [..., kv, D] in 32 bits at rows `at` of pages `where`."""
    k, v = s["kc"][where, :, at].to(F32), s["vc"][where, :, at].to(F32)
    if s["ks"] is not None:
        k, v = k * s["ks"][:, None], v * s["vs"][:, None]
    return k, v


def plain_prefix(s):
    page, ctx, first = s["page"], s["ctx"].long(), s["first"].tolist()
    heads, kv, dim = s["q"].shape[1], s["kc"].shape[1], s["kc"].shape[3]
    seqs, wide, group = ctx.numel(), s["widest"], heads // kv
    row, counts, live = rows_of(s)
    prefix = s["prefix"].tolist()
    lead = torch.repeat_interleave(s["prefix"].long(), s["first"].long().diff())     # of each sequence
    # what each sequence has of its own
    at = lead[:, None] + torch.arange(s["apart"], device=DEV)
    there = at < (ctx + counts)[:, None]
    where = s["table"].long().clamp(min=0).gather(1, (at // page).clamp(max=s["table"].shape[1] - 1))
    k, v = gathered(s, where, at % page)                     # [seqs, positions, kv, D]
    q = s["q"][row].to(F32) / math.sqrt(dim)                 # [seqs, wide, heads, D]
    q = q.view(seqs, wide, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs, kv, -1, dim)
    j = at - ctx[:, None]
    bit = (s["masks"][row][:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1
    sees = ((j[:, None, :] < 0) | ((bit == 1) & (j < counts[:, None])[:, None, :])) & there[:, None, :]
    mine = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()).view(seqs, kv, group, wide, -1)
    mine = mine.masked_fill(~sees[:, None, None], -math.inf).flatten(2, 3)           # [seqs, kv, rows, positions]
    # the prefix of each group, once for its sequences
    top, common = mine.amax(-1, keepdim=True), []
    for g, p in enumerate(prefix):
        b = slice(first[g], first[g + 1])
        x = torch.arange(p, device=DEV)
        pk, pv = gathered(s, s["table"][first[g]].long()[x // page], x % page)       # [positions, kv, D]
        rows = q[b].transpose(0, 1).reshape(kv, -1, dim)
        score = torch.matmul(rows, pk.permute(1, 2, 0).contiguous())
        common.append((score, pv))
        if p:
            m = score.amax(-1).view(kv, -1, q.shape[2]).transpose(0, 1)[..., None]
            top[b] = torch.maximum(top[b], m)
    top = torch.where(top == -math.inf, 0.0, top)
    w = torch.exp(mine - top)
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, v.transpose(1, 2).contiguous())
    for g, (score, pv) in enumerate(common):
        b = slice(first[g], first[g + 1])
        w = torch.exp(score - top[b].transpose(0, 1).reshape(kv, -1, 1))
        total[b] += w.sum(-1).view(kv, -1, q.shape[2]).transpose(0, 1)[..., None]
        o[b] += torch.matmul(w, pv.transpose(0, 1).contiguous()).view(kv, -1, q.shape[2], dim).transpose(0, 1)
    o = torch.where(total > 0, o / total, 0.0)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    spread_out = lambda x: x.view(seqs, kv, group, wide, -1).permute(0, 3, 1, 2, 4).reshape(seqs, wide, heads, -1)
    s["out"].copy_(spread_out(o)[live])
    s["lse"].copy_(spread_out(lse)[live][..., 0])
    return s["out"], s["lse"]


def plain_bounds(s):
    page = s["page"]
    old, new = s["old"].long() // page, s["new"].long() // page
    col = torch.arange(s["table"].shape[1], device=DEV)
    which = s["table"][(col >= old[:, None]) & (col < new[:, None])].long()
    k = s["kc"][:, which].to(F32)
    s["bounds"][:, which] = torch.stack((k.amin(3), k.amax(3)), 3).to(s["bounds"].dtype)
    return whole_values(s["bounds"])


def plain_select(s):
    case, page = s["case"], s["page"]
    count, kv, dim = case["count"], case["kv"], case["dim"]
    whole = s["ctx"].long() // page
    seqs, wide = whole.numel(), s["widest"]
    row, counts, live = rows_of(s)
    table = s["table"].long().clamp(min=0)
    col = torch.arange(table.shape[1], device=DEV)
    # scores in 64 bits: a block next to the border is in or out by its last digits
    q = s["q"][row].double().view(seqs, wide, kv, -1, dim)
    up, down = q.clamp(min=0).sum(3).permute(0, 2, 3, 1), q.clamp(max=0).sum(3).permute(0, 2, 3, 1)
    b = s["bounds"].to(F16 if case["cache"] == "e4m3" else s["bounds"].dtype)[table].double()   # [seqs, blocks, kv, 2, D]
    score = torch.matmul(b[:, :, :, 1].transpose(1, 2).contiguous(), up.contiguous())
    score += torch.matmul(b[:, :, :, 0].transpose(1, 2).contiguous(), down.contiguous())        # [seqs, kv, blocks, wide]
    score = score.permute(0, 3, 1, 2)
    edge = (col < case["first"]) | (col >= whole[:, None] - case["last"])
    score = torch.where(edge[:, None, None], math.inf, score)
    score = torch.where((col < whole[:, None])[:, None, None], score, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :count]
    rank = torch.arange(best.shape[-1], device=DEV)
    none = torch.iinfo(torch.int32).max
    best = torch.where(rank < whole[:, None, None, None], best, none).sort(-1)[0].to(torch.int32)
    best = torch.where(best == none, -1, best)
    s["out"].fill_(-1)
    s["out"][..., : best.shape[-1]] = best[live]
    return s["out"]


def plain_blocks(s):
    page, ctx = s["page"], s["ctx"].long()
    heads, kv, dim = s["q"].shape[1], s["kc"].shape[1], s["kc"].shape[3]
    start = s["start"].long()
    counts = start[1:] - start[:-1]
    seq = torch.repeat_interleave(torch.arange(ctx.numel(), device=DEV), counts)     # of each token
    table, whole = s["table"].long().clamp(min=0), ctx // page
    for part in torch.arange(s["q"].shape[0], device=DEV).split(64):
        b = seq[part]
        blocks = s["blocks"][part].long()                                            # [tokens, kv, count]
        inside = torch.arange(page, device=DEV)
        at = (blocks.clamp(min=0)[..., None] * page + inside).flatten(2)
        there = (blocks >= 0)[..., None].expand(-1, -1, -1, page).flatten(2)
        # the page where the context ends, and the tokens behind it
        tail = torch.arange(page + s["widest"], device=DEV) + (whole[b] * page)[:, None]
        j = tail - ctx[b][:, None]
        bit = (s["masks"][part][:, None] >> j.clamp(0, 63)) & 1
        sees = (j < 0) | ((bit == 1) & (j < counts[b][:, None]))
        at = torch.cat((at, tail[:, None].expand(-1, kv, -1)), 2)
        there = torch.cat((there, sees[:, None].expand(-1, kv, -1)), 2)
        where = table[b[:, None, None], (at // page).clamp(max=table.shape[1] - 1)]
        h = torch.arange(kv, device=DEV)[:, None]
        k, v = s["kc"][where, h, at % page].to(F32), s["vc"][where, h, at % page].to(F32)
        if s["ks"] is not None:
            k, v = k * s["ks"][:, None, None], v * s["vs"][:, None, None]
        q = s["q"][part].to(F32).view(-1, kv, heads // kv, dim) / math.sqrt(dim)
        score = torch.matmul(q, k.transpose(2, 3).contiguous()).masked_fill(~there[:, :, None], -math.inf)
        top = score.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        w = torch.exp(score - top)
        total = w.sum(-1, keepdim=True)
        o = torch.matmul(w, v)
        s["out"][part] = torch.where(total > 0, o / total, 0.0).flatten(1, 2).to(s["out"].dtype)
        s["lse"][part] = torch.where(total > 0, top + torch.log(total), -math.inf).flatten(1)
    return s["out"], s["lse"]


# ----------------------------------------------------------------------------------------------
# the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"prefix": exact_prefix, "bounds": exact_bounds, "select": exact_select, "blocks": exact_blocks}[case["op"]](s)


def attended(s, b, h, positions, tree, rows):
    """Output and log-sum of the query heads of key/value head h for tokens `rows` of sequence b, over these
    positions of it and over those of its tokens that `tree` (a truth value for each) lets them see."""
    q, page, n = s["q"], s["page"], tree.shape[1]
    kv, dim = s["kc"].shape[1], q.shape[2]
    each = q.shape[1] // kv
    at = torch.cat((positions, int(s["ctx"][b]) + torch.arange(n, device=DEV)))
    where = s["table"][b].long()[at // page]
    k, v = (x[where, h, at % page].double() for x in (s["kc"], s["vc"]))
    if s["ks"] is not None:
        k, v = k * s["ks"][h].double(), v * s["vs"][h].double()
    x = torch.matmul(q[rows, h * each: (h + 1) * each].double().reshape(-1, dim), k.T.contiguous()) / dim ** 0.5
    x = x.view(-1, each, at.numel())
    x[:, :, positions.numel():].masked_fill_(~tree[:, None], -math.inf)
    w = torch.nan_to_num(torch.softmax(x, -1))
    return torch.matmul(w.flatten(0, 1), v).view(-1, each, dim), torch.logsumexp(x, -1)


def empty_answer(s):
    return (torch.zeros(s["q"].shape, dtype=F64, device=DEV),
            torch.full(s["q"].shape[:2], -math.inf, dtype=F64, device=DEV))


def tree_of(s, t0, n):
    bits = s["masks"][t0: t0 + n, None] >> torch.arange(n, device=DEV)
    return (bits & 1) == 1


def exact_prefix(s):
    out, lse = empty_answer(s)
    start, kv = s["start"].tolist(), s["kc"].shape[1]
    each = s["q"].shape[1] // kv
    for b, c in enumerate(s["ctx"].tolist()):
        rows, n = slice(start[b], start[b + 1]), start[b + 1] - start[b]
        for h in range(kv if n else 0):
            hs = slice(h * each, (h + 1) * each)
            out[rows, hs], lse[rows, hs] = attended(s, b, h, torch.arange(c, device=DEV), tree_of(s, start[b], n), rows)
    return out, lse


def exact_bounds(s):
    want, page = torch.zeros(s["bounds"].shape, dtype=F16 if s["bounds"].dtype == E4M3 else s["bounds"].dtype, device=DEV), s["page"]
    table = s["table"].tolist()
    for b, (old, new) in enumerate(zip(s["old"].tolist(), s["new"].tolist())):
        which = torch.tensor(table[b][old // page: new // page], dtype=torch.long, device=DEV)
        for l in range(want.shape[0] if which.numel() else 0):
            keys = s["kc"][l, which].to(want.dtype).sort(2)[0]
            want[l, which] = keys[:, :, [0, -1]]
    return want.double()


def exact_select(s):
    case, page, kv = s["case"], s["page"], s["case"]["kv"]
    out = torch.full(s["out"].shape, -1, dtype=torch.int32, device=DEV)
    start, count = s["start"].tolist(), case["count"]
    for b, c in enumerate(s["ctx"].tolist()):
        whole = c // page
        pages = s["table"][b, :whole].long()
        for t in range(start[b], start[b + 1]) if whole else ():
            q = s["q"][t].double().view(kv, -1, 1, case["dim"])
            lo, hi = s["bounds"][pages].double().permute(2, 1, 0, 3)[:, :, None]    # [kv, 1, blocks, D]
            score = torch.maximum(q * lo, q * hi).sum(-1).sum(1)
            score[:, : case["first"]] = math.inf
            score[:, max(0, whole - case["last"]):] = math.inf
            m = min(count, whole)
            for h in range(kv):
                order = np.argsort(-score[h].cpu().numpy(), kind="stable")[:m]
                out[t, h, :m] = torch.from_numpy(np.sort(order).astype(np.int32)).to(DEV)
    return out


def exact_blocks(s):
    out, lse = empty_answer(s)
    start, kv, page = s["start"].tolist(), s["kc"].shape[1], s["page"]
    each = s["q"].shape[1] // kv
    inside = torch.arange(page, device=DEV)
    blocks = s["blocks"].cpu()
    for b, c in enumerate(s["ctx"].tolist()):
        n = start[b + 1] - start[b]
        tree = tree_of(s, start[b], n)
        end = torch.arange(c // page * page, c, device=DEV)
        for i in range(n):
            t = start[b] + i
            for h in range(kv):
                mine = [int(x) for x in blocks[t, h] if x >= 0]
                at = torch.cat([torch.tensor(mine, dtype=torch.long, device=DEV)[:, None].mul(page).add(inside).flatten(), end])
                hs = slice(h * each, (h + 1) * each)
                o, x = attended(s, b, h, at, tree[i: i + 1], slice(t, t + 1))
                out[t, hs], lse[t, hs] = o[0], x[0]
    return out, lse
