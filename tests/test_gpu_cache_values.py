"""Attention over the paged cache at the edges of its types, and with its contexts split: values that are
not finite, values and scores next to the largest numbers, positions in other waves and other pieces.

A context is split where a workspace is given and the table has room for more than SPLITS positions,
so the tables here are that long where a test wants pieces (columns behind a sequence's pages are -1).
"""
import math

import pytest

import ultra_bit_weight_uint32_amd as ubw
from test_gpu_cache import BF16, DEV, E4M3, F16, batch_of, cache_of, gen, i32, randn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
SPLITS = 768   # the longest context that is not split, of all sizes


def columns(page, split):
    """Columns a table needs at least so that contexts are split."""
    return SPLITS // page + 1 if split else 0


def attend(q, cache, table, start, ctx, masks=None, scale=None, split=False):
    """(out, lse), with every word of them and of the workspace set before the call."""
    t, heads, dim = q.shape
    tree = max(b - a for a, b in zip(start, start[1:]))
    ws = None
    if split:
        assert table.shape[1] * cache.page_size > SPLITS
        ws = ubw.tree_attn_workspace(len(ctx), tree, heads, cache.kv_heads, dim, DEV)
        ws.fill_(math.nan)
    out, lse = torch.full_like(q, 77.0), torch.full((t, heads), 77.0, device=DEV)
    ubw.tree_attn(q, cache, table, i32(start), i32(ctx), masks, max_tree=tree, scale=scale, out=out, lse=lse, workspace=ws)
    return out, lse


# ---------------------------------------------------------------------------------------------
# values that are not finite

@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16, E4M3], ids=str)
@pytest.mark.parametrize("tokens,heads", [(3, 2), (4, 8), (9, 6), (16, 8)], ids=str)
def test_tree_values_that_are_not_finite(tokens, heads, dtype, dim, split):
    """Each tree token in turn holds NaN (or infinity) in one dim of its value: the rows that see it get it
    there and nowhere else, the others are as they were. Contexts end in each of a workgroup's waves, so
    that the wave that meets it is not the one that writes the rows; 6 to 128 rows of a head."""
    page = 16
    ctx = [5, 40, 70, 100, 300]
    g = gen(dim + tokens)
    drafts = [tokens] * len(ctx)
    table, pages = batch_of(ctx, drafts, page, g, cols=columns(page, split))
    cache = cache_of(pages, 1, page, dim, dtype, g)
    t = tokens * len(ctx)
    q = randn((t, heads, dim), F16 if dtype is E4M3 else dtype, g)
    start = [tokens * i for i in range(len(ctx) + 1)]
    masks = torch.randint(0, 1 << tokens, (t,), device=DEV, generator=g)
    clean = attend(q, cache, table, start, ctx, masks, split=split)
    assert torch.isfinite(clean[0]).all()
    for j in sorted({0, tokens // 2, tokens - 1}):
        bad = math.nan if dtype is E4M3 or j % 2 else math.inf
        at = [(table[b, (c + j) // page].long(), (c + j) % page) for b, c in enumerate(ctx)]
        was = [cache.v[p, 0, r, 7].clone() for p, r in at]
        for p, r in at:
            cache.v[p, 0, r, 7] = bad
        want = clean[0].clone()
        want[((masks >> j) & 1) == 1, :, 7] = bad
        for _ in range(3):
            got = attend(q, cache, table, start, ctx, masks, split=split)
            assert torch.equal(got[0].nan_to_num(99.0, 98.0), want.nan_to_num(99.0, 98.0)), j
            assert torch.equal(got[1], clean[1])
        for (p, r), x in zip(at, was):
            cache.v[p, 0, r, 7] = x
