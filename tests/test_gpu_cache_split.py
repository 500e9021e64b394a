"""Attention over the paged cache with its contexts split over workgroups and joined: every tile, batches
larger than a workgroup, pieces of more than one unit, contents of device memory that are out of range.

A context is split where a workspace is given and the table has room for more positions than the largest
limit below; each test states its room, so that it cannot fall back to the single launch unnoticed.
"""
import math

import numpy as np
import pytest

import ultra_bit_weight_uint32_amd as ubw
from test_gpu_cache import (BF16, DEV, E4M3, F16, attention_reference, batch_of, cache_of, check_attention, gen, i32,
                            randn)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
SPLITS = 768   # the longest context that is not split, of all sizes
UNIT = 128     # positions that pieces are cut by


def split_call(q, cache, table, start, ctx, masks=None, tree=None, ws=None, **kw):
    t, heads, dim = q.shape
    assert table.shape[1] * cache.page_size > SPLITS
    tree = tree or max(b - a for a, b in zip(start, start[1:]))
    if ws is None:
        ws = ubw.tree_attn_workspace(len(ctx), tree, heads, cache.kv_heads, dim, DEV)
        ws.fill_(math.nan)
    out, lse = torch.full_like(q, 77.0), torch.full((t, heads), 77.0, device=DEV)
    ubw.tree_attn(q, cache, table, i32(start), i32(ctx), masks, max_tree=tree, out=out, lse=lse, workspace=ws, **kw)
    return out, lse


@pytest.mark.parametrize("rows", [(1, 1), (5, 3), (2, 8), (3, 10), (9, 4), (5, 12), (33, 2), (16, 8), (40, 5)], ids=str)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("qt,ct", [(F16, F16), (BF16, BF16), (F16, E4M3), (BF16, E4M3)], ids=str)
def test_every_tile_split(qt, ct, dim, rows):
    """1 to 200 rows of a key/value head (tokens x query heads of it), of each type and size; the call again
    gives the same bits."""
    tokens, group = rows
    g = gen(tokens * 10 + group + dim)
    ctx, drafts = [1111, 130, 0, 127, 390], [tokens, 1, tokens, max(1, tokens // 2), tokens]
    table, pages = batch_of(ctx, drafts, 16, g)
    cache = cache_of(pages, 2, 16, dim, ct, g, token_major=tokens % 2 == 1)
    start = [0] + list(np.cumsum(drafts))
    t = start[-1]
    q = randn((t, 2 * group, dim), qt, g)
    masks = torch.randint(-2 ** 63, 2 ** 63 - 1, (t,), device=DEV, generator=g)
    masks[-1] = -1
    masks[start[2]] = 0   # no context either: sees nothing
    first = split_call(q, cache, table, start, ctx, masks)
    check_attention(*first, attention_reference(q, cache, table, start, ctx, masks), qt, 1200)
    again = split_call(q, cache, table, start, ctx, masks)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("seqs,longest,kv,group", [(700, 900, 1, 1), (700, 900, 2, 10), (4096, 60, 1, 2), (300, 700, 2, 40)])
def test_batches_larger_than_a_workgroup_split(seqs, longest, kv, group):
    """More sequences than a workgroup has threads, up to as many as there may be; and more units than there
    are pieces, so that pieces have several, some sequences are cut and some are not."""
    g = gen(seqs + group)
    r = np.random.default_rng(seqs + kv)
    ctx = (longest * r.random(seqs) ** 3).astype(int).tolist()
    ctx[0], ctx[-1] = longest, longest
    drafts = r.integers(0, 3, seqs).tolist()
    drafts[0] = drafts[-1] = 2
    units = sum(kv * -(-(c + n) // UNIT) for c, n in zip(ctx, drafts) if n)
    assert units > 512
    table, pages = batch_of(ctx, drafts, 16, g, cols=49)
    cache = cache_of(pages, kv, 16, 64, BF16, g)
    start = [0] + list(np.cumsum(drafts))
    q = randn((start[-1], kv * group, 64), BF16, g)
    out, lse = split_call(q, cache, table, start, ctx)
    # (the reference of all rows takes minutes: these sequences, each as a batch of its own)
    for b in sorted({0, 1, 2, seqs // 2, seqs - 2, seqs - 1, *r.integers(0, seqs, 60).tolist()}):
        rows = slice(start[b], start[b + 1])
        if drafts[b]:
            want = attention_reference(q[rows], cache, table[b:b + 1], [0, drafts[b]], [ctx[b]], None)
            check_attention(out[rows], lse[rows], want, BF16, longest + 2)
    whole = torch.full_like(q, 77.0)
    ubw.tree_attn(q, cache, table, i32(start), i32(ctx), max_tree=2, out=whole)   # one launch, without pieces
    # each is within 2 half steps (2^-8) of its mean of values, and a little
    assert (out.float() - whole.float()).abs().max() <= 2.0 ** -6 * cache.v.float().abs().max()
    assert not (out == 77).any()


def test_a_workgroup_takes_several_pieces():
    """Pieces of 8 units and more, three for each workgroup: joined from up to a hundred."""
    g = gen(7)
    ctx, drafts = [90000, 100000], [2, 1]
    table, pages = batch_of(ctx, drafts, 256, g)
    for kv, group, dim, qt, ct in ((8, 1, 64, F16, F16), (8, 6, 128, BF16, BF16), (8, 2, 128, F16, E4M3)):
        cache = cache_of(pages, kv, 256, dim, ct, g)
        q = randn((3, kv * group, dim), qt, g)
        assert sum(-(-(c + n) // UNIT) for c, n in zip(ctx, drafts)) * kv > 512 * 8
        out, lse = split_call(q, cache, table, [0, 2, 3], ctx)
        for h in (0, kv * group - 1):   # of one query head, as a cache of one head
            hk = h // group
            one = ubw.KVCache(cache.k[:, hk:hk + 1].contiguous(), cache.v[:, hk:hk + 1].contiguous(),
                              *(None if s is None else s[hk:hk + 1].clone() for s in (cache.k_scale, cache.v_scale)))
            want = attention_reference(q[:, h:h + 1].contiguous(), one, table, [0, 2, 3], ctx, None)
            check_attention(out[:, h:h + 1], lse[:, h:h + 1], want, qt, 100001)


@pytest.mark.parametrize("heads,tree", [(4, 3), (40, 3), (80, 3)])
def test_what_is_out_of_range_split(heads, tree):
    """Lengths beyond the table, entries that are no pages, negative contexts, rows of no sequence, trees over
    max_tree, starts that do not ascend: cut as documented, nothing else written."""
    kv, dim, page, cols = 2, 64, 16, 60
    g = gen(15)
    cache = cache_of(70, kv, page, dim, F16, g)
    table = torch.randint(-3, 73, (4, cols), dtype=torch.int32, device=DEV, generator=g)
    table[0, 5:9] = i32([70, 2 ** 31 - 1, -2 ** 31, -1])
    table[3] = -1                                       # no page at all
    ctx, start = [700, 2 ** 31 - 1, -5, 900], [0, 2, 4, 7, 8]
    q = randn((10, heads, dim), F16, g)
    out, lse = split_call(q, cache, table, start, ctx, tree=tree)
    want = attention_reference(q[:8], cache, table, start, ctx, None)
    check_attention(out[:8], lse[:8], want, F16, cols * page)
    assert (out[8:] == 77).all() and (lse[8:] == 77).all()
    out, lse = split_call(q, cache, table, start, ctx, tree=2)
    assert (out[6] == 77).all() and not (out[5] == 77).any()   # the third token of a tree
    # starts that do not ascend, or pass the rows there are
    ws = ubw.tree_attn_workspace(4, tree, heads, kv, dim, DEV)
    guard = torch.full((10, heads, dim), 77.0, dtype=F16, device=DEV)
    ubw.tree_attn(q[:7], cache, table, i32([5, -3, 1000, 2, 7]), i32([2 ** 31 - 1, 0, -2 ** 31, 900]), max_tree=tree,
                  out=guard[:7], workspace=ws)
    assert (guard[7:] == 77).all()


def test_a_captured_split_call_beside_eager_ones():
    """A captured call of many rows, replayed with its lengths and table changed in place, between eager calls
    with a workspace of their own."""
    g = gen(17)
    heads, kv, dim, page = 16, 2, 128, 16
    table, pages = batch_of([2000, 900], [16, 16], page, g)
    cache = cache_of(pages, kv, page, dim, BF16, g)
    q, start, ctx = randn((32, heads, dim), BF16, g), i32([0, 16, 32]), i32([2000, 900])
    ws = [ubw.tree_attn_workspace(2, 16, heads, kv, dim, DEV) for _ in "ab"]
    args = dict(max_tree=16)
    ubw.tree_attn(q, cache, table, start, ctx, workspace=ws[0], **args)
    torch.cuda.synchronize()
    graph, out = torch.cuda.CUDAGraph(), torch.zeros_like(q)
    with torch.cuda.graph(graph):
        ubw.tree_attn(q, cache, table, start, ctx, out=out, workspace=ws[1], **args)
    shuffled = table.clone()
    shuffled[0, :100] = shuffled[0, :100].flip(0)
    for lens, tab in (([2000, 900], table.clone()), ([3, 1], shuffled), ([0, 890], shuffled), ([1999, 64], table.clone())):
        ctx.copy_(i32(lens))
        table.copy_(tab)
        out.fill_(77)
        graph.replay()
        eager = ubw.tree_attn(q, cache, table, start, ctx, workspace=ws[0], **args)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), lens


def test_masks_and_tables_in_their_other_forms():
    """A table whose rows lie apart, masks as uint64, queries and outputs that are parts of larger buffers, and
    outputs written over the queries: the results of the plain call."""
    g = gen(23)
    for tokens, heads, dt, dim in ((4, 8, F16, 128), (9, 40, BF16, 64), (3, 6, BF16, 256)):
        ctx, drafts, start = [1300, 77], [tokens, tokens], [0, tokens, 2 * tokens]
        table, pages = batch_of(ctx, drafts, 16, g)
        cache = cache_of(pages, 2, 16, dim, dt, g)
        q = randn((2 * tokens, heads, dim), dt, g)
        masks = torch.randint(-2 ** 63, 2 ** 63 - 1, (2 * tokens,), device=DEV, generator=g)
        want = split_call(q, cache, table, start, ctx, masks)
        apart = torch.nn.functional.pad(table, (2, 5), value=10 ** 6)[:, 2:-5]
        assert not apart.is_contiguous()
        for split in (True, False):
            ws = ubw.tree_attn_workspace(2, tokens, heads, 2, dim, DEV) if split else None
            wide = torch.zeros((2 * tokens, heads + 3, dim), dtype=dt, device=DEV)
            wide[:, 1:-2] = q
            got = ubw.tree_attn(wide[:, 1:-2], cache, apart, i32(start), i32(ctx), masks.view(torch.uint64), max_tree=tokens,
                                workspace=ws, out=torch.full_like(wide, 77)[:, 2:-1])
            plain = ubw.tree_attn(q, cache, table, i32(start), i32(ctx), masks, max_tree=tokens, workspace=ws)
            assert torch.equal(got, plain) and (not split or torch.equal(got, want[0]))
            over = q.clone()
            ubw.tree_attn(over, cache, table, i32(start), i32(ctx), masks, max_tree=tokens, workspace=ws, out=over)
            assert torch.equal(over, plain)


def test_a_thousand_heads_over_one():
    g = gen(24)
    table, pages = batch_of([900, 5], [1, 2], 16, g)
    for dt, ct in ((F16, E4M3), (BF16, BF16)):
        cache = cache_of(pages, 1, 16, 64, ct, g)
        q = randn((3, 1024, 64), dt, g)
        out, lse = split_call(q, cache, table, [0, 1, 3], [900, 5])
        for h in (0, 127, 128, 1023):
            want = attention_reference(q[:, h:h + 1].contiguous(), cache, table, [0, 1, 3], [900, 5], None)
            check_attention(out[:, h:h + 1], lse[:, h:h + 1], want, dt, 1000)
