"""Attention over selected blocks: bounds of pages' keys (exactly), the choice of blocks (exactly, against the definition
in 64 bits), attention over lists against 64 bits, and the calls together in a decoding loop.
"""
import math

import numpy as np
import pytest

import ultra_bit_weight_uint32_amd as ubw
from test_gpu_cache import (BF16, DEV, E4M3, F16, F32, F64, batch_of, cache_of, check_attention, gen, i32, randn)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def random_masks(t, g):
    m = torch.randint(-2 ** 63, 2 ** 63 - 1, (t,), device=DEV, generator=g)
    m[torch.rand(t, device=DEV, generator=g) < 0.2] = 0
    return m


# ---------------------------------------------------------------------------------------------
# bounds

def bits(x):
    """Values by what they stand for: NaN as one number, zeros of both signs alike."""
    return x.float().nan_to_num(12345.0, 1e30, -1e30) + 0.0


@pytest.mark.parametrize("page,kv,layers", [(16, 8, 3), (32, 1, 1), (64, 5, 2), (128, 2, 2), (1024, 3, 1)], ids=str)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16, E4M3], ids=str)
def test_bounds(dtype, dim, page, kv, layers):
    g = gen(page + dim + kv)
    start = [0, page - 1, 5, 3 * page, 2 * page, -7, 100 * page]
    stop = [3 * page, page, page - 1, 3 * page, 4 * page + 1, page, 2 ** 31 - 1]
    cols = 6
    pages = 7 * cols + 3
    order = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)
    table = order[:7 * cols].view(7, cols).contiguous()
    table[4, 3] = pages     # on no page
    table[0, 1] = table[4, 2]   # held by two
    shape = (layers, pages, kv, page, dim)
    if page == 64:   # token-major
        k = randn((layers, pages, page, kv, dim), dtype, g).transpose(2, 3)
    else:
        k = randn(shape, dtype, g)
    k[-1, 3, 0, 2, 5], k[0, :, -1, 7, 1] = math.nan, math.nan
    if dtype is not E4M3:
        k[0, 4, 0, 1, 2], k[0, 4, 0, 3, 3] = math.inf, -math.inf
    cache = ubw.KVCache(k if layers > 1 else k[0], k if layers > 1 else k[0])
    have = torch.full((layers, pages, kv, 2, dim), 3.0, device=DEV).to(dtype)
    want = have.float()
    named = torch.zeros(pages, dtype=torch.bool, device=DEV)
    for b in range(7):
        for c in range(max(start[b], 0) // page, min(max(stop[b], 0) // page, cols)):
            if 0 <= int(table[b, c]) < pages:
                named[table[b, c].long()] = True
    f = k.float()
    want[:, named] = torch.stack((f.amin(3), f.amax(3)), 3)[:, named]   # (torch's pass NaN on)
    assert named.sum() == 5   # three, one, none, none, one of them again, one
    for most in (0, 4 * page + 1):
        got = have.clone()
        ubw.page_bounds(cache, got if layers > 1 else got[0], table, i32(start), i32(stop), max_new=most)
        assert torch.equal(bits(got), bits(want))


@pytest.mark.parametrize("dtype,least", [(F16, 2.0 ** -24), (BF16, 2.0 ** -133), (E4M3, 2.0 ** -9)], ids=str)
def test_bounds_and_choice_of_the_smallest_values(dtype, least):
    """Multiples of the type's smallest value, which have no full mantissa."""
    g = gen(2)
    k = torch.randint(-7, 8, (6, 2, 16, 128), device=DEV, generator=g).double().mul(least).to(F32).to(dtype)
    cache = ubw.KVCache(k, k)
    got = torch.full((6, 2, 2, 128), 1.0, device=DEV).to(dtype)
    ubw.page_bounds(cache, got, i32([[3, 0, 1, 5, 2, 4]]), i32([0]), i32([96]))
    f = k.cpu().float()
    assert torch.equal(got.cpu().float(), torch.stack((f.amin(2), f.amax(2)), 2)) and got.float().ne(0).any()
    qt = F16 if dtype is E4M3 else dtype
    for tokens in (1, 3):
        q = torch.randint(-7, 8, (tokens, 4, 128), device=DEV, generator=g).double().mul(torch.finfo(qt).smallest_normal / 8)
        select_and_check(q.to(F32).to(qt), got, i32([[3, 0, 1, 5, 2, 4]]), [0, tokens], [96], 3, 16, 0, 0)


def test_bounds_of_many_pages():
    """More pages than the launch has groups of lanes, so that each takes several; far rows of a large cache."""
    g = gen(1)
    k = randn((1, 40000, 1, 16, 64), F16, g)
    cache = ubw.KVCache(k, k)
    table = torch.randperm(40000, device=DEV, generator=g).to(torch.int32).view(8, 5000)
    seqs = table.repeat(40, 1)    # all of them many times over
    got = torch.zeros((1, 40000, 1, 2, 64), dtype=F16, device=DEV)
    n = seqs.shape[0]
    ubw.page_bounds(cache, got, seqs, i32([0] * n), i32([5000 * 16] * n))
    assert torch.equal(got, torch.stack((k.amin(3), k.amax(3)), 3))
    dim, page, pages = 256, 1024, 9000   # 4.7 GB
    k = torch.empty((pages, 1, page, dim), dtype=F16, device=DEV)
    k[-1] = randn((1, page, dim), F16, g)
    got = torch.zeros((pages, 1, 2, dim), dtype=F16, device=DEV)
    ubw.page_bounds(ubw.KVCache(k, k), got, i32([[pages - 1]]), i32([0]), i32([page]))
    assert torch.equal(got[-1], torch.stack((k[-1].amin(1), k[-1].amax(1)), 1)) and not got[:-1].any()


# ---------------------------------------------------------------------------------------------
# the choice

def scores_of(q, bounds, table, whole, kv):
    """[kv, blocks] of one token, in 64 bits, as the definition has them; blocks on no page are -inf."""
    pages = bounds.shape[0]
    pg = table[:whole].long()
    ok = (pg >= 0) & (pg < pages)
    b = bounds.cpu().float().double()[pg.clamp(0, pages - 1)]          # [blocks, kv, 2, D]
    x = q.double().view(kv, -1, 1, q.shape[-1])                         # [kv, G, 1, D]
    lo, hi = b[:, :, 0].transpose(0, 1)[:, None], b[:, :, 1].transpose(0, 1)[:, None]
    s = torch.where(x < 0, x * lo, x * hi)
    s = torch.where(x == 0, 0.0, torch.where(x.isnan() | lo.isnan(), math.nan, s)).sum(-1).sum(1)
    return s, ok


def choose(s, ok, count, first, last):
    """Indices of the chosen blocks of one head, ascending."""
    n = s.numel()
    if n <= count:
        return list(range(n))
    key = [(1 if first <= i < n - last else 0, 0 if ok[i] else 1, 0 if math.isnan(s[i]) else 1,
            -(0.0 if math.isnan(s[i]) else float(s[i])), i) for i in range(n)]
    return sorted(k[-1] for k in sorted(key)[:count])


def select_and_check(q, bounds, table, start, ctx, count, page, first=1, last=1, tree=None, exact=True, **kw):
    t, heads, dim = q.shape
    kv = bounds.shape[1]
    tree = tree or max(1, max(b - a for a, b in zip(start, start[1:])))
    ws = ubw.block_select_workspace(t, kv, table.shape[1], DEV)
    ws.fill_(-1)
    out = torch.full((t, kv, count), 77, dtype=torch.int32, device=DEV)
    got = ubw.block_select(q, bounds, table, i32(start), i32(ctx), count, page_size=page, first=first, last=last, max_tree=tree,
                           out=out, workspace=ws, **kw)
    assert got is out
    qc, tc = q.cpu().float(), table.cpu()
    want = torch.full((t, kv, count), 77, dtype=torch.int32)
    for b, c in enumerate(ctx):
        whole = min(max(c, 0) // page, table.shape[1])
        for r in range(start[b], min(start[b + 1], start[b] + tree)):
            s, ok = scores_of(qc[r], bounds, tc[b], whole, kv)
            for h in range(kv):
                at = choose(s[h], ok, count, first, last)
                want[r, h] = torch.tensor(at + [-1] * (count - len(at)), dtype=torch.int32)
    bad = (out.cpu() != want).any(-1).nonzero()
    assert bad.numel() == 0, (bad[:5].tolist(), [out[tuple(i)].tolist() for i in bad[:2]], [want[tuple(i)].tolist() for i in bad[:2]])
    return out


def bounds_of(pages, kv, dim, dtype, g):
    mid, half = randn((pages, kv, 1, dim), F32, g), randn((pages, kv, 1, dim), F32, g).abs()
    return torch.cat((mid - half, mid + half), 2).to(dtype)


SELECT = [  # heads, kv, dim, q type, bounds type, page, contexts, tokens, count, first, last
    (1, 1, 64, F16, F16, 16, [3200], [1], 7, 0, 0), (8, 8, 128, BF16, BF16, 32, [5000, 31, 32, 0, 700], [1] * 5, 16, 1, 2),
    (16, 2, 128, F16, E4M3, 16, [2000, 100, 16 * 12 + 3], [1, 0, 1], 12, 2, 3), (12, 4, 64, BF16, E4M3, 64, [9000], [1], 1, 0, 0),
    (24, 1, 256, F16, F16, 16, [1600, 999], [1, 1], 20, 5, 5), (5, 5, 256, BF16, E4M3, 128, [20000, 640], [1, 1], 33, 0, 4),
    (8, 2, 128, F16, F16, 16, [1700, 0, 300, 4000], [3, 2, 16, 1], 9, 1, 1), (16, 2, 64, BF16, BF16, 32, [3000, 1000], [33, 17], 8, 0, 2),
    (6, 3, 256, F16, E4M3, 16, [900, 16], [2, 64], 30, 3, 0), (8, 1, 128, BF16, E4M3, 16, [5003], [40], 50, 2, 2),
    (4, 4, 256, BF16, BF16, 1024, [70000], [5], 17, 1, 1), (40, 1, 128, F16, F16, 16, [500], [4], 31, 10, 21),
    (10, 5, 64, F16, E4M3, 16, [777, 130], [18, 3], 4, 1, 0),
]


@pytest.mark.parametrize("case", SELECT, ids=str)
def test_choice(case):
    heads, kv, dim, qt, bt, page, ctx, drafts, count, first, last = case
    g = gen(heads + dim + sum(ctx))
    table, pages = batch_of(ctx, drafts, page, g)
    bounds = bounds_of(pages, kv, dim, bt, g)
    start = [0] + list(np.cumsum(drafts))
    t = start[-1]
    q = randn((t + 1, heads + 2, dim), qt, g)[:t, 1:-1] if heads % 4 == 0 else randn((t, heads, dim), qt, g)
    a = select_and_check(q, bounds, table, start, ctx, count, page, first, last)
    b = select_and_check(q, bounds, table, start, ctx, count, page, first, last, max_len=max(ctx))
    c = select_and_check(q, bounds, table, start, ctx, count, page, first, last, max_len=max(x + n for x, n in zip(ctx, drafts)))
    assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("tokens", [1, 3])
@pytest.mark.parametrize("blocks,count", [(4095, 100), (4096, 4000), (4097, 1), (4100, 37), (9001, 2000), (70000, 513)])
def test_choice_of_many_blocks(blocks, count, tokens):
    """Around and beyond the scores that a workgroup keeps; half of the blocks are copies of others."""
    g = gen(blocks + count)
    table = torch.randint(0, 5000, (1, blocks), dtype=torch.int32, device=DEV, generator=g)
    table[0, blocks // 2:] = table[0, :blocks - blocks // 2].clone()
    q = randn((tokens, 2, 64), F16, g)
    select_and_check(q, bounds_of(5000, 1, 64, F16, g), table, [0, tokens], [blocks * 16 + 5], count, 16, *((2, 3) if count > 5 else (0, 0)))


@pytest.mark.parametrize("kv,tokens,seqs", [(32, 1, 33), (8, 16, 9), (64, 2, 8)], ids=str)
def test_choice_for_many_rows(kv, tokens, seqs):
    """Short contexts of many tokens and heads, up to and beyond 128 blocks; equal scores, NaN and blocks on no page."""
    g = gen(kv)
    bounds = bounds_of(40, kv, 64, F16, g)
    bounds[7, 0, 0, 3] = bounds[7, 0, 1, 3] = math.nan
    start = [tokens * b for b in range(seqs + 1)]
    q = randn((seqs * tokens, kv, 64), F16, g)
    for cols in (63, 128, 129):
        table = torch.randint(-1, 41, (seqs, cols), dtype=torch.int32, device=DEV, generator=g)
        ctx = [min((b * 47) % 140, cols) * 16 + b % 16 for b in range(seqs)]
        for count, first, last in ((1, 0, 0), (20, 1, 2), (60, 30, 30)):
            select_and_check(q, bounds, table, start, ctx, count, 16, first, last)
            if count == 20:
                select_and_check(q, bounds, table, start, ctx, count, 16, first, last, tree=max(1, tokens - 1), max_len=max(ctx))


@pytest.mark.parametrize("cols", [256, 257, 512, 513, 1024, 1025])
def test_choice_for_many_rows_of_longer_contexts(cols):
    """8 trees of 16 tokens, 32 heads: two contexts of the whole table and nearly so, the others short."""
    g = gen(cols)
    bounds = bounds_of(60, 32, 64, F16, g)
    bounds[7, 0, 0, 3] = bounds[7, 0, 1, 3] = math.nan
    table = torch.randint(-1, 61, (8, cols), dtype=torch.int32, device=DEV, generator=g)
    ctx = [cols * 16, 30, 0, (cols - 70) * 16 + 3, 500, 16 * 16, 16 * 17, 2 ** 31 - 1 if cols < 500 else 7]
    q = randn((128, 32, 64), F16, g)
    for count, first, last in ((16, 1, 2), (70, 0, 0)):
        select_and_check(q, bounds, table, [16 * b for b in range(9)], ctx, count, 16, first, last)


@pytest.mark.parametrize("tokens", [1, 17])
@pytest.mark.parametrize("blocks", [100, 600, 5000])
def test_equal_scores_go_to_the_lowest_index(blocks, tokens):
    """All equal, a few values, zeros of both signs, and all but one or two equal."""
    g = gen(blocks)
    dim, pages = 128, 8
    bounds = torch.zeros((pages, 1, 2, dim), dtype=F16, device=DEV)
    bounds[:, :, 1] = 1.0
    bounds[1] = -0.0
    bounds[2, 0, 1, 3] = 2.0
    q = torch.ones((tokens, 1, dim), dtype=F16, device=DEV)
    for pick in ([3], [3, 4, 5], [3, 2, 6], [1, 0], [1]):
        table = i32(pick)[torch.randint(0, len(pick), (1, blocks), device=DEV, generator=g)]
        for count in (1, 50, blocks - 1, blocks):
            select_and_check(q, bounds, table, [0, tokens], [blocks * 16], count, 16, 0, 0)
    table = i32([[3] * blocks])
    table[0, blocks // 2] = 2
    select_and_check(q, bounds, table, [0, tokens], [blocks * 16], 3, 16, 0, 1)
    q.zero_()                     # every score is 0, of either sign
    q[:, :, 1::2] = -0.0
    select_and_check(q, bounds, i32([[1, 2, 0, 3] * (blocks // 4)]), [0, tokens], [blocks // 4 * 64], 5, 16, 0, 0)


@pytest.mark.parametrize("tokens", [1, 5])
def test_choice_of_unusual_values(tokens):
    """Bounds and queries that are infinite or NaN, blocks on no page, contexts beyond the table, rows of no sequence and
    behind max_tree, starts out of range."""
    g = gen(6)
    page, dim, kv, heads = 16, 128, 2, 6
    bounds = bounds_of(50, kv, dim, F16, g)
    bounds[7, 0, 0, 3] = bounds[7, 0, 1, 3] = math.nan
    bounds[8, 1, 1, 5] = math.inf
    bounds[9, :, 0, 9] = -math.inf
    table = torch.randint(-2, 53, (3, 60), dtype=torch.int32, device=DEV, generator=g)
    table[0, 4:8] = i32([7, 8, 9, 2 ** 31 - 1])
    ctx, start = [60 * page, 2 ** 31 - 1, 17 * page + 3], [0, tokens, 2 * tokens, 3 * tokens]
    q = randn((3 * tokens + 2, heads, dim), F16, g)
    q[0, :, 9] = q[0, :, 9].abs()   # with an upper bound that is finite the block is as others
    select_and_check(q, bounds, table, start, ctx, 9, page, 1, 1)
    if tokens > 1:
        select_and_check(q, bounds, table, start, ctx, 9, page, 0, 0, tree=tokens - 2)
    q[1, 0, 0] = math.nan           # every block of that head: the lowest indices
    q[2, 5, 1] = math.inf
    select_and_check(q, bounds, table, start, ctx, 9, page, 0, 0)
    cut = ubw.block_select(q, bounds, table, i32(start), i32(ctx), 5, page_size=page, max_tree=tokens, max_len=10 * page,
                           workspace=ubw.block_select_workspace(3 * tokens + 2, kv, 60, DEV),
                           out=torch.full((3 * tokens + 2, kv, 5), 77, dtype=torch.int32, device=DEV))
    assert (cut[:3 * tokens] <= 10).all() and (cut[3 * tokens:] == 77).all()
    ws = ubw.block_select_workspace(4, kv, 60, DEV)
    guard = torch.full((ws.numel() + 64,), 7, dtype=torch.int64, device=DEV)
    over = torch.full((8, kv, 5), 77, dtype=torch.int32, device=DEV)
    for starts in ([2, -3, 1000, 4], [4, 0, 4, 0], [-5, 9, 2, 3]):
        ubw.block_select(q[:4], bounds, table, i32(starts), i32([2 ** 31 - 1, -5, 900]), 5, page_size=page, max_tree=64,
                         workspace=guard[:ws.numel()], out=over[:4])
        torch.cuda.synchronize()
        assert (over[4:] == 77).all() and (guard[ws.numel():] == 7).all()


# ---------------------------------------------------------------------------------------------
# attention over lists

def lists_of(ctx, drafts, kv, count, page, g, spare=0):
    """int32 [tokens, kv, count]: ascending blocks of each token's context, -1 behind them."""
    rng = np.random.default_rng(int(torch.randint(0, 2 ** 31, (1,), device=DEV, generator=g)))
    rows = []
    for c, n in zip(ctx, drafts):
        whole = max(c, 0) // page
        for _ in range(n):
            one = np.full((kv, count), -1, np.int32)
            for h in range(kv):
                m = min(whole, int(rng.integers(0, count + 1)) if rng.random() < 0.3 else count)
                one[h, :m] = np.sort(rng.permutation(whole)[:m])
            rows.append(one)
    return torch.from_numpy(np.stack(rows)).to(DEV)


def block_reference(q, cache, table, start, ctx, blocks, masks, scale=None):
    """out, lse in 64 bits, and what the tolerance is made of (as tree attention's reference)."""
    q = q.double().cpu()
    t, heads, dim = q.shape
    kv, page = cache.kv_heads, cache.page_size
    scale = dim ** -0.5 if scale is None else scale
    k, v = cache.k.cpu().float().double(), cache.v.cpu().float().double()
    if cache.k_scale is not None:
        k = k * cache.k_scale.double().cpu()[:, None, None]
    if cache.v_scale is not None:
        v = v * cache.v_scale.double().cpu()[:, None, None]
    out, size = torch.zeros_like(q), torch.zeros_like(q)
    lse, reach = torch.full((t, heads), -math.inf, dtype=F64), torch.zeros((t, heads), dtype=F64)
    table, blocks = table.cpu(), blocks.cpu()
    cols = table.shape[1]
    masks = None if masks is None else [int(m) & (2 ** 64 - 1) for m in masks.tolist()]
    for b, c in enumerate(ctx):
        c, n = max(c, 0), start[b + 1] - start[b]
        whole = c // page
        for i in range(n):
            r = start[b] + i
            tree = (1 << (i + 1)) - 1 if masks is None else masks[r]
            tail = list(range(whole * page, c)) + [c + j for j in range(min(n, 64)) if tree >> j & 1]
            for hk in range(kv):
                at, before = [], -1
                for x in blocks[r, hk].tolist():
                    if x <= before or x >= min(whole, cols):
                        break
                    at += range(x * page, (x + 1) * page)
                    before = x
                at = torch.tensor([p for p in at + tail if p // page < cols], dtype=torch.long)
                pg = table[b, at // page].long()
                ok = (pg >= 0) & (pg < cache.pages)
                pg, row = pg[ok], (at % page)[ok]
                if not pg.numel():
                    continue
                kk, vv = k[pg, hk, row], v[pg, hk, row]
                for h in range(hk * heads // kv, (hk + 1) * heads // kv):
                    s = scale * (kk @ q[r, h])
                    w = torch.softmax(s, 0)
                    lse[r, h] = torch.logsumexp(s, 0)
                    out[r, h], size[r, h] = w @ vv, w @ vv.abs()
                    reach[r, h] = scale * (kk.abs() @ q[r, h].abs()).max()
    return out, lse, size, reach


def attend(q, cache, table, start, ctx, blocks, masks=None, split=True, tree=None, **kw):
    t, heads, dim = q.shape
    ws = None
    if split:
        ws = ubw.block_attn_workspace(t, heads, cache.kv_heads, dim, DEV)
        ws.fill_(math.nan)
    out, lse = torch.full_like(q, 77.0), torch.full((t, heads), 77.0, device=DEV)
    ubw.block_attn(q, cache, table, i32(start), i32(ctx), blocks, masks,
                   max_tree=tree or max(1, max(b - a for a, b in zip(start, start[1:]))), out=out, lse=lse, workspace=ws, **kw)
    return out, lse


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("group", [1, 3, 8, 16, 17, 40])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("qt,ct", [(F16, F16), (BF16, BF16), (F16, E4M3), (BF16, E4M3)], ids=str)
def test_attention_over_lists(qt, ct, dim, group, split):
    g = gen(dim + group)
    page = 16 if group % 2 else 32
    ctx, drafts = [700, 40, 0, 16, 333, 5], [2, 1, 3, 1, 5, 0]
    table, pages = batch_of(ctx, drafts, page, g)
    cache = cache_of(pages, 2, page, dim, ct, g, token_major=group == 3)
    start = [0] + list(np.cumsum(drafts))
    q = randn((start[-1], 2 * group, dim), qt, g)
    masks = random_masks(start[-1], g)
    masks[start[2]] = 0   # no context, no mask: sees nothing
    blocks = lists_of(ctx, drafts, 2, 14, page, g)
    got = attend(q, cache, table, start, ctx, blocks, masks, split)
    check_attention(*got, block_reference(q, cache, table, start, ctx, blocks, masks), qt, 600)
    again = attend(q, cache, table, start, ctx, blocks, masks, split)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("tokens", [1, 2, 64])
def test_lists_of_pages(tokens, page):
    """Contexts that end next to the borders of pages; single tokens, small and the largest trees."""
    g = gen(page + tokens)
    ctx = [0, 1, page - 1, page, page + 1, 3 * page - 1, 3 * page]
    drafts = [tokens] * 4 + [1] * 3
    table, pages = batch_of(ctx, drafts, page, g)
    cache = cache_of(pages, 1, page, 128, F16, g)
    start = [0] + list(np.cumsum(drafts))
    q = randn((start[-1], 4, 128), F16, g)
    blocks = lists_of(ctx, drafts, 1, 2, page, g)
    for m in (None, random_masks(start[-1], g)):
        got = attend(q, cache, table, start, ctx, blocks, m)
        check_attention(*got, block_reference(q, cache, table, start, ctx, blocks, m), F16, 4 * page)


def test_long_lists():
    """One token over 200 blocks of a long context, split over workgroups, and lists longer than a wave."""
    g = gen(4)
    for kv, group, dim, qt, ct, page, ctx, drafts, count in ((2, 8, 128, BF16, BF16, 16, [20000], [1], 200),
                                                            (1, 4, 64, F16, E4M3, 64, [30000, 9000], [1, 3], 130),
                                                            (1, 24, 128, F16, F16, 32, [9000], [4], 65)):
        table, pages = batch_of(ctx, drafts, page, g)
        cache = cache_of(pages, kv, page, dim, ct, g)
        start = [0] + list(np.cumsum(drafts))
        q = randn((start[-1], kv * group, dim), qt, g)
        blocks = lists_of(ctx, drafts, kv, count, page, g)
        got = attend(q, cache, table, start, ctx, blocks)
        check_attention(*got, block_reference(q, cache, table, start, ctx, blocks, None), qt, count * page + page + 64)


def test_lists_end_where_they_do_not_ascend():
    """... or name no whole block: no block counts twice and nothing is read that is not there."""
    g = gen(5)
    page, ctx, drafts = 16, [100, 2 ** 31 - 1, 40], [5, 2, 1]
    cache = cache_of(30, 1, page, 64, F16, g)
    table = torch.randint(-2, 33, (3, 8), dtype=torch.int32, device=DEV, generator=g)
    table[0] = torch.arange(8)
    start = [0, 5, 7, 8]
    q = randn((10, 2, 64), F16, g)
    blocks = i32([[0, 2, 2, 3], [3, 1, 4, 5], [-1, 1, 2, 3], [1, 5, 6, 7], [2 ** 31 - 1, 0, 1, 2], [0, 7, 8, 9], [-2 ** 31, 0, 1, 2],
                  [0, 1, 2, 3], [0, 1, 2, 3], [0, 1, 2, 3]])[:, None].contiguous()
    for split in (True, False):
        out, lse = attend(q, cache, table, start, ctx, blocks, split=split)
        want = block_reference(q[:8], cache, table, start, ctx, blocks[:8], None)
        check_attention(out[:8], lse[:8], want, F16, 200)
        assert (out[8:] == 77).all() and (lse[8:] == 77).all()   # rows of no sequence
        out, lse = attend(q, cache, table, start, ctx, blocks, split=split, tree=4)
        assert (out[4] == 77).all() and not (out[3] == 77).any()   # behind max_tree
        none = attend(q, cache, table, start, ctx, blocks[:, :, :0].contiguous(), split=split)
        want = block_reference(q[:8], cache, table, start, ctx, blocks[:8, :, :0], None)
        check_attention(none[0][:8], none[1][:8], want, F16, 200)
    ws = ubw.block_attn_workspace(4, 2, 1, 64, DEV)
    guard = torch.full((ws.numel() + 64,), 7.0, device=DEV)
    over = torch.full((8, 2, 64), 77.0, dtype=F16, device=DEV)
    for starts in ([2, -3, 1000, 4], [4, 0, 4, 0], [-5, 9, 2, 3]):
        ubw.block_attn(q[:4], cache, table, i32(starts), i32([2 ** 31 - 1, -5, 900]), blocks[:4], max_tree=64,
                       workspace=guard[:ws.numel()], out=over[:4])
        torch.cuda.synchronize()
        assert (over[4:] == 77).all() and (guard[ws.numel():] == 7).all()


@pytest.mark.parametrize("dtype", [F16, BF16, E4M3], ids=str)
def test_blocks_that_are_not_chosen_reach_nothing(dtype):
    """NaN in every block that is not chosen, behind the end and in unseen tokens of the tree."""
    g = gen(11)
    page, ctx, drafts = 16, [230, 70], [4, 1]
    table, pages = batch_of(ctx, drafts, page, g)
    cache = cache_of(pages, 1, page, 128, dtype, g)
    q = randn((5, 8, 128), F16 if dtype is E4M3 else dtype, g)
    blocks = i32([[1, 4, 9, -1]] * 4 + [[0, 2, -1, -1]])[:, None].contiguous()
    masks = torch.tensor([1, 3, 5, 9, 1], device=DEV)   # each its own token and the first
    masks[1:3] = 0
    start = [0, 4, 5]
    clean = attend(q, cache, table, start, ctx, blocks, masks)
    used = torch.zeros((pages, page), dtype=torch.bool, device=DEV)
    for b, rows in ((0, [0, 3]), (1, [0])):
        chosen = [int(x) for x in blocks[start[b], 0] if x >= 0]
        seen = [p for x in chosen for p in range(x * page, x * page + page)]
        seen += list(range(ctx[b] // page * page, ctx[b])) + [ctx[b] + j for j in rows]
        for p in seen:
            used[table[b, p // page].long(), p % page] = True
    bad = ~used[:, None, :, None].expand(cache.k.shape)
    for x in (cache.k, cache.v):
        x.copy_(torch.where(bad, torch.full_like(x.float(), math.nan), x.float()).to(dtype))
    got = attend(q, cache, table, start, ctx, blocks, masks)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    cache.v[table[0, (ctx[0] + 3) // page].long(), 0, (ctx[0] + 3) % page, 6] = math.nan   # seen by token 3 alone
    nan = torch.zeros_like(got[0], dtype=torch.bool)
    nan[3, :, 6] = True
    got = attend(q, cache, table, start, ctx, blocks, masks)
    assert torch.equal(got[0].isnan(), nan) and torch.equal(got[0][~nan], clean[0][~nan])


# ---------------------------------------------------------------------------------------------
# together

@pytest.mark.parametrize("dtype", [F16, E4M3], ids=str)
def test_a_decoding_loop(dtype):
    """A prompt, then steps of single tokens and trees: pages reserved, keys and values stored, bounds of the pages that
    filled, blocks chosen, attention over them. With room for all blocks it is tree attention; with less, the
    chosen blocks are those of the definition and the outputs those over them."""
    g = gen(30)
    page, kv, heads, dim, seqs = 16, 2, 8, 128, 3
    pool = ubw.page_pool(pages=120, page_size=page, seqs=seqs, max_pages=40)
    ks = torch.full((kv,), 0.03, device=DEV) if dtype is E4M3 else None
    k, v = (torch.zeros((120, kv, page, dim), device=DEV).to(dtype) for _ in "kv")
    cache = ubw.KVCache(k, v, ks, ks)
    bounds = torch.zeros((120, kv, 2, dim), dtype=dtype, device=DEV)
    freq = (10000.0 ** (-torch.arange(0, dim, 2, device=DEV, dtype=F64) / dim)).to(F32)
    length = [0] * seqs
    count = 8
    for step, new in enumerate(([300, 17, 150], [1, 1, 1], [4, 16, 1], [1, 1, 1], [16, 0, 30], [1, 1, 1])):
        new = [min(n, 64) if step else n for n in new]
        ubw.pages_reserve(pool, i32(new))
        where = torch.cat([torch.arange(a, a + n) for a, n in zip(length, new)])
        row = torch.repeat_interleave(torch.arange(seqs), torch.tensor(new))
        slots = pool.table[row.to(DEV), (where // page).to(DEV)] * page + (where % page).to(DEV)
        t = where.numel()
        x = [randn((t, h, dim), F32, g) for h in (heads, kv, kv)]
        q = ubw.qk_norm_rope(*x, cache, where.to(torch.int32).to(DEV), slots.to(torch.int32), freq, out_dtype=F16)
        start = [0] + list(np.cumsum(new))
        if step:
            args = (pool.table, i32(start), i32(length))
            tree = max(new)
            ws = ubw.block_select_workspace(t, kv, 40, DEV)
            got = select_and_check(q, bounds, pool.table, start, length, count, page, 1, 2)
            out, lse = attend(q, cache, pool.table, start, length, got)
            check_attention(out, lse, block_reference(q, cache, pool.table, start, length, got, None), F16, 400)
            every = ubw.block_select(q, bounds, *args, 40, page_size=page, max_tree=tree, workspace=ws)
            all_out, all_lse = attend(q, cache, pool.table, start, length, every)
            dense = torch.zeros_like(q)
            dense_lse = torch.zeros((t, heads), device=DEV)
            ubw.tree_attn(q, cache, *args, max_tree=tree, out=dense, lse=dense_lse)
            # both within half a step of fp16 and their weights' roundings (2^-11 each) of a mean of values below 6
            assert (all_out.float() - dense.float()).abs().max() <= 4 * 2.0 ** -11 * 6
            # the same scores, up to 400 weights summed in fp32 in another order: 2 (400 + 64) V + 8 V (|lse| + 16) < 1e-4, V = 2^-24
            assert (all_lse - dense_lse).abs().max() <= 1e-4
        after = [a + n for a, n in zip(length, new)]
        ubw.pages_trim(pool, i32(after))
        ubw.page_bounds(cache, bounds, pool.table, i32(length), pool.len, max_new=max(new))
        length = after
        whole = pool.table[0, :length[0] // page].long()
        f = k[whole].float()
        assert torch.equal(bounds[whole].float(), torch.stack((f.amin(2), f.amax(2)), 2))
    assert int(pool.status) == 0


def test_captured_and_concurrent_calls():
    """The three calls captured in one graph, replayed with lengths, table and cache changed in place; two streams with
    workspaces of their own at once; buffers of other strides."""
    g = gen(31)
    page, kv, heads, dim, count = 16, 2, 16, 128, 12
    ctx, drafts = [2000, 900, 50], [4, 1, 7]
    table, pages = batch_of([2600, 1500, 200], drafts, page, g)
    cache = cache_of(pages, kv, page, dim, BF16, g)
    start = i32([0, 4, 5, 12])
    q, masks = randn((12, heads, dim), BF16, g), random_masks(12, g)
    cols = table.shape[1]

    def step(lens, old, bounds, blocks, out, ws):
        ubw.page_bounds(cache, bounds, table, old, lens)
        ubw.block_select(q, bounds, table, start, lens, count, page_size=page, max_tree=7, workspace=ws[0], out=blocks)
        return ubw.block_attn(q, cache, table, start, lens, blocks, masks, max_tree=7, workspace=ws[1], out=out)

    def buffers():
        return (torch.zeros((pages, kv, 2, dim), dtype=BF16, device=DEV), torch.zeros((12, kv, count), dtype=torch.int32, device=DEV),
                torch.zeros_like(q), (ubw.block_select_workspace(12, kv, cols, DEV), ubw.block_attn_workspace(12, heads, kv, dim, DEV)))

    lens, zero = i32(ctx), i32([0, 0, 0])
    eager, held = buffers(), buffers()
    want = step(lens, zero, *eager).clone()
    graph = torch.cuda.CUDAGraph()
    step(lens, zero, *held)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(lens, zero, *held)
    for new in (ctx, [2599, 3, 0], [0, 16, 190], [1999, 1400, 17]):
        lens.copy_(i32(new))
        table[0, :100] = table[0, :100].flip(0)
        cache.k[3].add_(0.5)
        held[2].fill_(77)
        graph.replay()
        again = step(lens, zero, *eager)
        torch.cuda.synchronize()
        assert torch.equal(held[2], again) and torch.equal(held[1], eager[1]), new
    lens.copy_(i32(ctx))
    want = step(lens, zero, *eager).clone()
    streams, sets = [torch.cuda.Stream() for _ in "ab"], [buffers() for _ in "ab"]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, b in zip(streams, sets):
            with torch.cuda.stream(s):
                step(lens, zero, *b)
    torch.cuda.synchronize()
    assert all(torch.equal(b[2], want) for b in sets)
    wide = torch.zeros((12, heads + 3, dim), dtype=BF16, device=DEV)
    wide[:, 1:-2] = q
    apart = torch.nn.functional.pad(table, (2, 5), value=10 ** 6)[:, 2:-5]
    got = ubw.block_select(wide[:, 1:-2], eager[0], apart, start, lens, count, page_size=page, max_tree=7, workspace=eager[3][0])
    assert torch.equal(got, eager[1])
    got = ubw.block_attn(wide[:, 1:-2], cache, apart, start, lens, got, masks.view(torch.uint64), max_tree=7, workspace=eager[3][1],
                         out=torch.full_like(wide, 77)[:, 2:-1])
    assert torch.equal(got, want)


def test_arguments():
    g = gen(1)
    ctx, drafts = [70, 5], [1, 1]
    table, pages = batch_of(ctx, drafts, 16, g)
    cache = cache_of(pages, 2, 16, 64, F16, g)
    q, bounds = randn((2, 4, 64), F16, g), torch.zeros((pages, 2, 2, 64), dtype=F16, device=DEV)
    common = dict(q=q, table=table, q_start=i32([0, 1, 2]), ctx_len=i32(ctx), max_tree=1)
    sel = common | dict(bounds=bounds, count=2, page_size=16, workspace=ubw.block_select_workspace(2, 2, table.shape[1], DEV))
    assert ubw.block_select(**sel).shape == (2, 2, 2)
    for bad, error in ((dict(bounds=bounds[0]), ValueError), (dict(bounds=bounds.float()), TypeError), (dict(bounds=bounds.cpu()), ValueError),
                       (dict(bounds=bounds.to(BF16)), ubw.UbwError), (dict(count=0), ubw.UbwError), (dict(first=2), ubw.UbwError),
                       (dict(workspace=None), ubw.UbwError), (dict(workspace=sel["workspace"][:-1]), ubw.UbwError),
                       (dict(q=q.float()), TypeError), (dict(page_size=20), ubw.UbwError),
                       (dict(out=torch.zeros((2, 2, 3), dtype=torch.int32, device=DEV)), ValueError),
                       (dict(bounds=bounds.transpose(0, 1)), (ValueError, ubw.UbwError))):
        with pytest.raises(error):
            ubw.block_select(**(sel | bad))
    blocks = torch.zeros((2, 2, 1), dtype=torch.int32, device=DEV)
    att = common | dict(cache=cache, blocks=blocks)
    assert ubw.block_attn(**att).shape == q.shape
    for bad, error in ((dict(blocks=blocks[:1]), ValueError), (dict(blocks=blocks[:, :1].contiguous()), ValueError),
                       (dict(blocks=blocks.long()), TypeError), (dict(blocks=blocks[:, :, 0].contiguous()), ValueError),
                       (dict(q=q.to(BF16)), ubw.UbwError)):
        with pytest.raises(error):
            ubw.block_attn(**(att | bad))
    assert ubw.block_attn(**(att | dict(q=q[:0], q_start=i32([0, 0, 0]), blocks=blocks[:0]))).shape == (0, 4, 64)
    old, new = i32([0, 0]), i32([64, 0])
    ubw.page_bounds(cache, bounds, table, old, new)
    for bad, error in ((dict(bounds=bounds.to(BF16)), TypeError), (dict(bounds=bounds[None]), ValueError), (dict(stop=new[:1]), ValueError),
                       (dict(start=old.long()), TypeError), (dict(bounds=bounds.cpu()), ValueError)):
        with pytest.raises(error):
            ubw.page_bounds(**(dict(cache=cache, bounds=bounds, table=table, start=old, stop=new) | bad))
