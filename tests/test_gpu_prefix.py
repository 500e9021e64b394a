"""Attention over shared prefixes against 64 bits and against tree attention: groups of every kind, every tile and type,
prefixes cut into many pieces, contents of device memory that are out of range, captured and concurrent calls.

The reference reads every sequence's context by its own table row, so a prefix read from another row is right only if
it is the same keys and values; tolerances are those of tree attention (two parts are joined as its pieces are).
"""
import math

import numpy as np
import pytest

import ultra_bit_weight_uint32_amd as ubw
from test_gpu_cache import (BF16, DEV, E4M3, F16, attention_reference, cache_of, check_attention, gen, i32, randn)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def shared_batch(first, prefix, own, drafts, page, kv, dim, dtype, g, token_major=False, cols=0, spare=2):
    """(cache, table, ctx): the sequences of group g hold the whole pages of its prefix together, and a copy each
    of the page on which it ends, as forks do. first: first sequence of each group and the end (sequences
    outside have prefixes of their own of 0)."""
    n = len(own)
    lead, pre = list(range(n)), [0] * n
    for k, p in enumerate(prefix):
        for b in range(first[k], first[k + 1]):
            lead[b], pre[b] = first[k], p
    ctx = [p + o for p, o in zip(pre, own)]
    need = [-(-(c + d) // page) for c, d in zip(ctx, drafts)]
    width = max(max(need), cols, 1)
    table = np.full((n, width), -1, np.int32)
    at, copies = 0, []
    mine = [max(need[b], -(-pre[b] // page)) if lead[b] == b else need[b] - min(need[b], pre[b] // page) for b in range(n)]
    pages = sum(mine) + spare
    order = torch.randperm(pages, device=DEV, generator=g).cpu().numpy().astype(np.int32)
    for b in range(n):
        keep = 0 if lead[b] == b else min(need[b], pre[b] // page)
        table[b, :keep] = table[lead[b], :keep]
        table[b, keep:keep + mine[b]] = order[at:at + mine[b]]
        at += mine[b]
        if lead[b] != b and pre[b] % page and need[b] > keep:
            copies.append((table[lead[b], keep], table[b, keep]))
    cache = cache_of(pages, kv, page, dim, dtype, g, token_major=token_major)
    for x, y in copies:
        for c in (cache.k, cache.v):
            c[int(y)].copy_(c[int(x)])
    return cache, torch.from_numpy(table).to(DEV), ctx


def wide_of(table, cache):
    """The table with columns on no page, so many that contexts could be long ones: short ones are not shared."""
    position = 2 * cache.kv_heads * cache.head_dim * cache.k.element_size()
    cols = (100 << 20) // (position * table.shape[0] * cache.page_size) + 1
    return torch.nn.functional.pad(table, (0, max(cols - table.shape[1], 0)), value=-1)


def call(q, cache, table, start, ctx, first, prefix, masks=None, tree=None, ws=None, scale=None, wide=True, **kw):
    t, heads, dim = q.shape
    table = wide_of(table, cache) if wide else table
    tree = tree or max(1, max(b - a for a, b in zip(start, start[1:])))
    if ws is None:
        ws = ubw.prefix_attn_workspace(len(ctx), len(prefix), t, tree, heads, cache.kv_heads, dim, DEV)
        ws.fill_(math.nan)   # scratch: what it held does not matter
    out, lse = torch.full_like(q, 77.0), torch.full((t, heads), 77.0, device=DEV)
    ubw.prefix_attn(q, cache, table, i32(start), i32(ctx), i32(first), i32(prefix), masks, max_tree=tree, out=out, lse=lse,
                    workspace=ws, scale=scale, **kw)
    return out, lse


def random_masks(t, g):
    m = torch.randint(-2 ** 63, 2 ** 63 - 1, (t,), device=DEV, generator=g)
    m[torch.rand(t, device=DEV, generator=g) < 0.2] = 0
    return m


@pytest.mark.parametrize("rows", [(1, 1), (1, 8), (5, 3), (3, 11), (2, 16), (9, 4), (33, 2), (16, 8), (40, 5)], ids=str)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("qt,ct", [(F16, F16), (BF16, BF16), (F16, E4M3), (BF16, E4M3)], ids=str)
def test_every_tile(qt, ct, dim, rows):
    """1 to 200 rows of a sequence and key/value head, groups of one to five sequences and some in none, prefixes that
    are a multiple of 16 and that are not, members without tokens (the first among them) and without positions of
    their own. The call again gives the same bits."""
    tokens, group = rows
    g = gen(tokens * 10 + group + dim)
    first, prefix = [1, 4, 5, 10], [203, 150, 64]
    own = [300, 5, 0, 77, 40, 1, 130, 20, 0, 64, 0]
    drafts = [tokens, tokens, 1, max(1, tokens // 2), tokens, 0, tokens, 1, tokens, tokens, tokens]
    cache, table, ctx = shared_batch(first, prefix, own, drafts, 16, 2, dim, ct, g, token_major=tokens % 2 == 1)
    start = [0] + list(np.cumsum(drafts))
    q = randn((start[-1], 2 * group, dim), qt, g)
    masks = random_masks(start[-1], g)
    masks[start[10]] = 0   # no context, no mask: sees nothing
    got = call(q, cache, table, start, ctx, first, prefix, masks)
    want = attention_reference(q, cache, table, start, ctx, masks)
    check_attention(*got, want, qt, 500)
    short = call(q, cache, table, start, ctx, first, prefix, masks, max_len=max(c + n for c, n in zip(ctx, drafts)))
    check_attention(*short, want, qt, 500)   # (that short, nothing is shared)
    again = call(q, cache, table, start, ctx, first, prefix, masks)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("page", [16, 32, 128, 1024])
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 31, 128, 129, 1025])
def test_ends_of_prefixes(prefix, page):
    """Prefixes that end next to the borders of tiles, pages and units, with and without positions behind them."""
    g = gen(page + prefix)
    own, drafts = [0, 1, 15, 130], [1, 3, 1, 2]
    cache, table, ctx = shared_batch([0, 4], [prefix], own, drafts, page, 2, 128, BF16, g)
    start = [0] + list(np.cumsum(drafts))
    q = randn((start[-1], 8, 128), BF16, g)
    got = call(q, cache, table, start, ctx, [0, 4], [prefix])
    check_attention(*got, attention_reference(q, cache, table, start, ctx, None), BF16, 1300)


def test_a_prefix_is_read_from_one_row():
    """Whole tiles of a prefix are read by the row of the first sequence that has tokens: the others' entries do not
    matter; a prefix longer than a context counts as that context; below 0, as 0."""
    g = gen(3)
    page, prefix = 32, 160
    own, drafts = [0, 9, 33, 4], [0, 2, 1, 5]
    cache, table, ctx = shared_batch([0, 4], [prefix], own, drafts, page, 2, 64, F16, g)
    start = [0] + list(np.cumsum(drafts))
    q = randn((8, 6, 64), F16, g)
    want = attention_reference(q, cache, table, start, ctx, None)
    holes = table.clone()
    holes[0] = -1               # has no tokens: not even its row is read
    holes[2:, :prefix // page] = 10 ** 6
    check_attention(*call(q, cache, holes, start, ctx, [0, 4], [prefix]), want, F16, 300)
    # two sequences share 100 positions and hold others behind them; a prefix said to be longer is cut
    ctx2 = [ctx[0], 96, ctx[2], ctx[3]]
    want = attention_reference(q, cache, table, start, ctx2, None)
    for said in (2 ** 31 - 1, 160, 96):
        check_attention(*call(q, cache, table, start, ctx2, [0, 4], [said]), want, F16, 300)
    for said in (-1, -2 ** 31):
        a, b = call(q, cache, table, start, ctx2, [0, 4], [said]), call(q, cache, table, start, ctx2, [0], [])
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("seqs,groups,kv,group,longest", [(300, 4, 2, 10, 700), (700, 300, 1, 1, 200), (1500, 700, 2, 2, 90),
                                                         (4096, 4096, 1, 1, 40), (4096, 1, 1, 2, 60)])
def test_batches_larger_than_a_workgroup(seqs, groups, kv, group, longest):
    """More sequences and groups than the planning workgroup has threads, up to as many as there may be."""
    g = gen(seqs + groups)
    r = np.random.default_rng(seqs + kv)
    first = [0] + sorted(r.choice(np.arange(1, seqs), groups - 1, replace=False).tolist()) + [seqs]
    prefix = r.integers(0, longest, groups).tolist()
    prefix[0] = longest
    own = (longest * r.random(seqs) ** 3).astype(int).tolist()
    drafts = r.integers(0, 3, seqs).tolist()
    drafts[0] = drafts[-1] = 2
    cache, table, ctx = shared_batch(first, prefix, own, drafts, 16, kv, 64, BF16, g)
    start = [0] + list(np.cumsum(drafts))
    q = randn((start[-1], kv * group, 64), BF16, g)
    out, lse = call(q, cache, table, start, ctx, first, prefix)
    # (the reference of all rows takes minutes: these sequences, each as a batch of its own)
    for b in sorted({0, 1, 2, seqs // 2, seqs - 2, seqs - 1, *r.integers(0, seqs, 60).tolist()}):
        rows = slice(start[b], start[b + 1])
        if drafts[b]:
            want = attention_reference(q[rows], cache, table[b:b + 1], [0, drafts[b]], [ctx[b]], None)
            check_attention(out[rows], lse[rows], want, BF16, 2 * longest + 2)
    whole = torch.full_like(q, 77.0)
    ubw.tree_attn(q, cache, table, i32(start), i32(ctx), max_tree=2, out=whole)
    # each is within 2 half steps (2^-8) of its mean of values, and a little
    assert (out.float() - whole.float()).abs().max() <= 2.0 ** -6 * cache.v.float().abs().max()
    assert not (out == 77).any()


@pytest.mark.parametrize("kv,ct,kinds", [(10, E4M3, [(8, 39, 32), (8, 20, 62), (8, 4, 31)]), (4, E4M3, [(8, 92, 54), (8, 36, 64), (4, 2, 215)]),
                                         (10, E4M3, [(8, 47, 44), (8, 11, 66), (8, 22, 23)]), (10, E4M3, [(8, 18, 61), (8, 60, 37), (8, 100, 44)]),
                                         (4, BF16, [(4, 74, 100), (8, 4, 64), (8, 18, 111)])], ids=str)
def test_batches_of_a_few_lengths(kv, ct, kinds):
    """Batches of two or three lengths (tokens, units of 128 positions, sequences): many rests of one cost, dealt out where
    the beginnings of several workgroups' runs fall together (computed by each workgroup in 32 bits, the last three left lists
    out). Every row is written, near tree attention's; some are held against 64 bits."""
    g = gen(kv + kinds[0][1])
    group, dim, page = 5, 128, 64
    r = np.random.default_rng(kv)
    each = [(n, u) for n, u, seqs in kinds for _ in range(seqs)]
    each = [each[i] for i in r.permutation(len(each))]
    most = max(u for _, u in each)
    ctx = [128 * u - n - int(r.integers(0, 128 - n)) for n, u in each]
    start = [0] + list(np.cumsum([n for n, _ in each]))
    cache = cache_of(300, kv, page, dim, ct, g)   # sequences have pages in common here and there
    table = torch.randint(0, 300, (len(ctx), 2 * most), dtype=torch.int32, device=DEV, generator=g)
    q = randn((int(start[-1]), kv * group, dim), BF16, g)
    out, lse = call(q, cache, table, start, ctx, [0], [], wide=False)
    whole, whole_lse = torch.empty_like(q), torch.empty_like(lse)
    ubw.tree_attn(q, cache, table, i32(start), i32(ctx), max_tree=8, out=whole, lse=whole_lse)
    # each is within 2 half steps (2^-8) of its mean of values, and a little; values are multiplied by less than 1.5
    assert (out.float() - whole.float()).abs().max() <= 2.0 ** -6 * 1.5 * cache.v.float().abs().max()
    # sums in fp32 over up to 128 `most` positions: relatively within (positions + 64) 2^-24 of the exact ones, each score
    # within (dim + 20) 2^-24 of scale sum |q||k| < 64, and the logarithm 4 2^-24 (|lse| + 16)
    assert (lse - whole_lse).abs().max() <= 2 * 2.0 ** -24 * (128 * most + 64 + 148 * 64 + 4 * 80)
    for b in r.integers(0, len(ctx), 3):
        rows = slice(start[b], start[b + 1])
        for h in (0, kv * group - 1):
            hk = h // group
            one = ubw.KVCache(cache.k[:, hk:hk + 1].contiguous(), cache.v[:, hk:hk + 1].contiguous(),
                              *(None if s is None else s[hk:hk + 1].clone() for s in (cache.k_scale, cache.v_scale)))
            want = attention_reference(q[rows, h:h + 1], one, table[b:b + 1], [0, each[b][0]], [ctx[b]], None)
            check_attention(out[rows, h:h + 1], lse[rows, h:h + 1], want, BF16, 128 * most)


@pytest.mark.parametrize("kv,group,dim,qt,ct", [(2, 8, 128, BF16, BF16), (1, 3, 64, F16, F16), (2, 8, 128, BF16, E4M3),
                                                (1, 4, 256, F16, F16), (2, 1, 128, F16, E4M3)], ids=str)
def test_long_prefixes(kv, group, dim, qt, ct):
    """Prefixes of many pieces, several to a workgroup, beside short ones, of several row blocks each."""
    g = gen(dim + group)
    first, prefix = [0, 9, 10, 14], [30007, 500, 9000]
    own = [0, 3000, 17, 1, 400, 0, 5, 90, 1000, 7, 300, 0, 20, 2]
    drafts = [3, 1, 2, 16, 1, 5, 1, 1, 4, 1, 33, 1, 2, 6]
    cache, table, ctx = shared_batch(first, prefix, own, drafts, 64, kv, dim, ct, g)
    start = [0] + list(np.cumsum(drafts))
    q = randn((start[-1], kv * group, dim), qt, g)
    masks = random_masks(start[-1], g)
    out, lse = call(q, cache, table, start, ctx, first, prefix, masks)
    for h in sorted({0, kv * group - 1}):   # of one query head, as a cache of one head
        hk = h // group
        one = ubw.KVCache(cache.k[:, hk:hk + 1].contiguous(), cache.v[:, hk:hk + 1].contiguous(),
                          *(None if s is None else s[hk:hk + 1].clone() for s in (cache.k_scale, cache.v_scale)))
        want = attention_reference(q[:, h:h + 1].contiguous(), one, table, start, ctx, masks)
        check_attention(out[:, h:h + 1], lse[:, h:h + 1], want, qt, 34000)


def test_what_is_out_of_range():
    """Lengths beyond the table, entries that are no pages, rows of no sequence, trees over max_tree: as in tree
    attention. Starts and groups that do not ascend, or overlap, write nothing else."""
    kv, dim, page, cols, heads = 2, 64, 16, 60, 6
    g = gen(15)
    cache = cache_of(70, kv, page, dim, F16, g)
    table = torch.randint(-3, 73, (4, cols), dtype=torch.int32, device=DEV, generator=g)
    table[0, 5:9] = i32([70, 2 ** 31 - 1, -2 ** 31, -1])
    table[1:3] = table[0]
    table[3] = -1                                       # no page at all
    ctx, start = [700, 2 ** 31 - 1, 400, 900], [0, 2, 4, 7, 8]
    q = randn((10, heads, dim), F16, g)
    out, lse = call(q, cache, table, start, ctx, [0, 3], [2 ** 31 - 1], tree=3)
    want = attention_reference(q[:8], cache, table, start, ctx, None)
    check_attention(out[:8], lse[:8], want, F16, cols * page)
    assert (out[8:] == 77).all() and (lse[8:] == 77).all()
    out, lse = call(q, cache, table, start, ctx, [0, 3], [400], tree=2)
    assert (out[6] == 77).all() and not (out[5] == 77).any()   # the third token of a tree
    check_attention(out[:6], lse[:6], tuple(x[:6] for x in want), F16, cols * page)
    ws = ubw.prefix_attn_workspace(4, 5, 7, 3, heads, kv, dim, DEV)
    guard = torch.full((ws.numel() + 64,), 7.0, device=DEV)
    table = wide_of(table, cache)
    for groups in ([0, 4, 0, 4, 0, 4], [4, 3, 2, 1, 0, 0], [-5, 9, 2, 3, 100, 2 ** 31 - 1], [0, 0, 0, 0, 0, 4]):
        for starts in ([0, 2, 4, 6, 7], [5, -3, 1000, 2, 7], [7, 0, 7, 0, 7]):
            guard.fill_(7.0)
            over = torch.full((10, heads, dim), 77.0, dtype=F16, device=DEV)
            ubw.prefix_attn(q[:7], cache, table, i32(starts), i32([2 ** 31 - 1, 0, -2 ** 31, 900]), i32(groups),
                            i32([300, 2 ** 31 - 1, -1, 16, 40]), max_tree=3, out=over[:7], workspace=guard[:ws.numel()])
            torch.cuda.synchronize()
            assert (over[7:] == 77).all() and (guard[ws.numel():] == 7).all()
    # starts that do not ascend share nothing: those of tree attention
    starts, lens = i32([5, 2, 4, 6, 7]), i32([200, 200, 200, 200])
    a = ubw.prefix_attn(q[:7], cache, table, starts, lens, i32([0, 4]), i32([160]), max_tree=3, workspace=ws, out=torch.zeros_like(q[:7]))
    b = ubw.prefix_attn(q[:7], cache, table, starts, lens, i32([0]), i32([]), max_tree=3, workspace=ws, out=torch.zeros_like(q[:7]))
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F16, BF16, E4M3], ids=str)
def test_values_that_are_not_finite(dtype):
    """NaN behind a sequence's end, in unseen tokens of a tree and in other pages reach nothing; in a seen token of a tree
    they reach those who see it; in the prefix everyone."""
    g = gen(8)
    page, dim, heads = 16, 128, 8
    first, prefix = [0, 3], [90]
    own, drafts = [3, 30, 0], [4, 1, 6]
    cache, table, ctx = shared_batch(first, prefix, own, drafts, page, 1, dim, dtype, g, spare=3)
    start = [0] + list(np.cumsum(drafts))
    qt = F16 if dtype is E4M3 else dtype
    q = randn((11, heads, dim), qt, g)
    masks = torch.randint(0, 64, (11,), device=DEV, generator=g)
    masks[:4] &= ~2     # token 1 of the first tree is seen by no one
    masks[5:] &= ~16    # and token 4 of the last by its own fifth alone
    masks[10] |= 16
    clean = call(q, cache, table, start, ctx, first, prefix, masks)
    used = torch.zeros((cache.pages, page), dtype=torch.bool, device=DEV)
    for b in range(3):
        for p in range(ctx[b] + drafts[b]):
            if not (b == 0 and p == ctx[0] + 1):
                used[table[b, p // page].long(), p % page] = True
    bad = ~used[:, None, :, None].expand(cache.k.shape)
    for x in (cache.k, cache.v):
        x.copy_(torch.where(bad, torch.full_like(x.float(), math.nan), x.float()).to(dtype))
    got = call(q, cache, table, start, ctx, first, prefix, masks)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    at = ctx[2] + 4
    cache.v[table[2, at // page].long(), 0, at % page, 7] = math.nan
    got = call(q, cache, table, start, ctx, first, prefix, masks)
    nan = torch.zeros_like(got[0], dtype=torch.bool)
    nan[10, :, 7] = True
    assert torch.equal(got[0].isnan(), nan) and torch.equal(got[0][~nan], clean[0][~nan])
    cache.v[table[0, 2].long(), 0, 5, 9] = math.nan   # position 37
    nan[:, :, 9] = True
    got = call(q, cache, table, start, ctx, first, prefix, masks)
    assert torch.equal(got[0].isnan(), nan) and torch.equal(got[0][~nan], clean[0][~nan])


@pytest.mark.parametrize("size", [2.0 ** 120, 2.0 ** 126])
def test_large_bf16_values(size):
    """Values whose sums pass fp32's range where their means do not: those of values 2^-100 as large, times 2^100."""
    g = gen(9)
    first, prefix, own, drafts = [0, 4], [2000], [3, 500, 0, 64], [1, 2, 16, 1]
    cache, table, ctx = shared_batch(first, prefix, own, drafts, 16, 1, 64, BF16, g)
    start = [0] + list(np.cumsum(drafts))
    q = randn((20, 8, 64), BF16, g)
    cache.v.clamp_(-1, 1).mul_(size)
    got = call(q, cache, table, start, ctx, first, prefix)
    assert torch.isfinite(got[0]).all()
    cache.v.mul_(2.0 ** -100)
    small = call(q, cache, table, start, ctx, first, prefix)
    # as two calls whose weights are rounded apart: 2^-8 of the mean of |v| <= size each, and of the result
    assert ((got[0].double() - small[0].double() * 2.0 ** 100).abs() <= 4 * 2.0 ** -8 * size).all()
    # scores are the same, but sums that passed the range are taken again under other maxima: each log-sum is within
    # (positions + 64) V + 4 V (|lse| + 16) of theirs, V = 2^-24 (sums in fp32; the logarithm and the product behind it)
    tol = 2 * 2.0 ** -24 * (2600 + 64 + 4 * (small[1].abs() + 16))
    assert ((got[1] - small[1]).abs() <= tol).all()


def test_streams_graphs_and_devices():
    """Two streams with workspaces of their own at once; a captured call replayed with its lengths, prefixes and table
    changed in place, between eager ones; any buffers' strides."""
    g = gen(17)
    heads, kv, dim, page = 16, 2, 128, 16
    first, prefix, own, drafts = [0, 3, 6], [700, 250], [100, 0, 30, 5, 60, 7], [4, 1, 2, 16, 1, 1]
    cache, table, ctx = shared_batch(first, prefix, own, drafts, page, kv, dim, BF16, g)
    start = [0] + list(np.cumsum(drafts))
    q = randn((25, heads, dim), BF16, g)
    want = call(q, cache, table, start, ctx, first, prefix)
    ws = [ubw.prefix_attn_workspace(6, 2, 25, 16, heads, kv, dim, DEV) for _ in "abc"]
    args = [i32(x) for x in (start, ctx, first, prefix)]
    table = wide_of(table, cache)
    streams, outs = [torch.cuda.Stream() for _ in "ab"], [torch.zeros_like(q) for _ in "ab"]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, o, w in zip(streams, outs, ws):
            with torch.cuda.stream(s):
                ubw.prefix_attn(q, cache, table, *args, max_tree=16, workspace=w, out=o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) for o in outs)
    wide = torch.zeros((25, heads + 3, dim), dtype=BF16, device=DEV)
    wide[:, 1:-2] = q
    apart = torch.nn.functional.pad(table, (2, 5), value=10 ** 6)[:, 2:-5]
    got = ubw.prefix_attn(wide[:, 1:-2], cache, apart, *args, max_tree=16, workspace=ws[0], out=torch.full_like(wide, 77)[:, 2:-1])
    assert torch.equal(got, want[0])
    graph, out = torch.cuda.CUDAGraph(), torch.zeros_like(q)
    with torch.cuda.graph(graph):
        ubw.prefix_attn(q, cache, table, *args, max_tree=16, out=out, workspace=ws[1])
    for lens, pre in ((ctx, prefix), ([700, 710, 705, 250, 255, 251], [700, 240]), ([0, 3, 1, 0, 2, 16], [16, 16]), (ctx, [0, 100])):
        args[1].copy_(i32(lens))
        args[3].copy_(i32(pre))
        out.fill_(77)
        graph.replay()
        eager = ubw.prefix_attn(q, cache, table, *args, max_tree=16, workspace=ws[0])
        torch.cuda.synchronize()
        assert torch.equal(out, eager), lens


@pytest.mark.parametrize("qt,ct,heads,kv,dim", [(F16, F16, 16, 2, 128), (BF16, E4M3, 8, 8, 64), (F16, E4M3, 24, 2, 256)], ids=str)
def test_short_contexts_are_those_of_tree_attention(qt, ct, heads, kv, dim):
    """... bit by bit; where the caller says that they are short, too, and up to the order of summing where not."""
    g = gen(23)
    first, prefix, own, drafts = [0, 3, 6], [700, 250], [100, 0, 30, 5, 60, 7, 9], [4, 1, 2, 16, 1, 0, 1]
    cache, table, ctx = shared_batch(first, prefix, own, drafts, 32, kv, dim, ct, g)
    start = [0] + list(np.cumsum(drafts))
    q = randn((25, heads, dim), qt, g)
    masks = random_masks(25, g)
    out, lse = torch.full_like(q, 77.0), torch.full((25, heads), 77.0, device=DEV)
    ws = ubw.tree_attn_workspace(7, 16, heads, kv, dim, DEV)
    ubw.tree_attn(q, cache, table, i32(start), i32(ctx), masks, max_tree=16, out=out, lse=lse, workspace=ws)
    want = attention_reference(q, cache, table, start, ctx, masks)
    check_attention(out, lse, want, qt, 900)
    got = call(q, cache, table, start, ctx, first, prefix, masks, wide=False)
    assert torch.equal(got[0], out) and torch.equal(got[1], lse)
    ubw.tree_attn(q, cache, wide_of(table, cache), i32(start), i32(ctx), masks, max_tree=16, max_len=820, out=out, lse=lse, workspace=ws)
    got = call(q, cache, table, start, ctx, first, prefix, masks, max_len=820)
    assert torch.equal(got[0], out) and torch.equal(got[1], lse)
    check_attention(*call(q, cache, table, start, ctx, first, prefix, masks), want, qt, 900)


def test_arguments():
    g = gen(1)
    cache, table, ctx = shared_batch([0, 2], [40], [1, 2], [1, 1], 16, 2, 64, F16, g)
    q = randn((2, 4, 64), F16, g)
    ws = ubw.prefix_attn_workspace(2, 1, 2, 1, 4, 2, 64, DEV)
    good = dict(q=q, cache=cache, table=table, q_start=i32([0, 1, 2]), ctx_len=i32(ctx), group_start=i32([0, 2]),
                prefix_len=i32([40]), max_tree=1, workspace=ws)
    assert ubw.prefix_attn(**good).shape == q.shape
    for bad, error in ((dict(group_start=i32([0, 1, 2])), ValueError), (dict(prefix_len=torch.tensor([40], device=DEV)), TypeError),
                       (dict(group_start=torch.tensor([0, 2], dtype=torch.int32)), ValueError), (dict(workspace=None), ubw.UbwError),
                       (dict(workspace=ws[:-1]), ubw.UbwError), (dict(q=q.float()), TypeError), (dict(q_start=i32([0, 2])), ValueError)):
        with pytest.raises(error):
            ubw.prefix_attn(**(good | bad))
    empty = ubw.prefix_attn(**(good | dict(q=q[:0], q_start=i32([0, 0, 0]))))
    assert empty.shape == (0, 4, 64)
