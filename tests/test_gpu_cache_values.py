"""Attention over the paged cache at the edges of its types, and with its contexts split: values that are
not finite, values and scores next to the largest numbers, positions in other waves and other pieces.

A context is split where a workspace is given and the table has room for more than SPLITS positions,
so the tables here are that long where a test wants pieces (columns behind a sequence's pages are -1).
"""
import math

import pytest

import ultra_bit_weight_uint32_amd as ubw
from test_gpu_cache import (BF16, DEV, E4M3, F16, attention_reference, batch_of, cache_of, check_attention, gen, i32,
                            near, randn, rope_reference)

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


# ---------------------------------------------------------------------------------------------
# large scores

APART = [(100, 101), (101, 100), (100, 132), (132, 100), (40, 700), (700, 40), (3, 1290), (1290, 3)]


def score_cache(dtype, dim, scores, g):
    """A one-head cache and a query row such that position p's score (scale 1) is exactly scores[p]: whole
    numbers below 2^11 in one dim, where the query has 1, and multiples of 2^27 over 16 dims of 2^15 x 2^8."""
    page, n = 16, len(scores)
    table, pages = batch_of([n - 1], [1], page, g, cols=columns(page, True))
    cache = cache_of(pages, 1, page, dim, dtype, g, scales=False)
    q = torch.zeros(dim, device=DEV)
    q[:16], q[20] = 2.0 ** 15, 8.0
    k = torch.zeros((n, dim), device=DEV)
    for p, x in enumerate(scores):
        k[p, :16] = 256.0 * round(x / 2 ** 27)
        k[p, 20] = (x - 2 ** 27 * round(x / 2 ** 27)) / 8
    assert torch.equal(k.to(dtype).float(), k)
    at = torch.arange(n, device=DEV)
    cache.k[table[0, at // page].long(), 0, at % page] = k.to(dtype)
    v = cache.v[table[0, at // page].long(), 0, at % page].double().cpu()
    return cache, table, q, v


@pytest.mark.parametrize("heads", [1, 20, 40, 100])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16, E4M3], ids=str)
def test_large_scores_weigh_by_their_difference(dtype, dim, heads):
    """Scores of 2^27 and 2^27 - 8, both exact in fp32, at positions of one tile, of two waves and of two
    pieces: they weigh 1 : e^-8, wherever they lie. The scores are exact, so an output is off by the
    weights' roundings (half a step of the type; e^-8 itself by under 2^-19), those of the sums and
    divisions (under 64 of fp32), and its own rounding."""
    qt = BF16 if dtype is E4M3 else dtype
    u = torch.finfo(qt).eps / 2
    g = gen(dim + heads)
    for hi, lo in APART:
        scores = [0] * (max(hi, lo) + 4)
        scores[hi], scores[lo] = 2 ** 27, 2 ** 27 - 8
        cache, table, q, v = score_cache(dtype, dim, scores, g)
        q = q.to(qt).expand(1, heads, dim).contiguous()
        w = math.exp(-8)
        want, size = (v[hi] + w * v[lo]) / (1 + w), (v[hi].abs() + w * v[lo].abs()) / (1 + w)
        off = (u + 2.0 ** -18 + 64 * 2.0 ** -24) * size
        tol = off + u * (want.abs() + off)
        for split in (True, False):
            out, lse = attend(q, cache, table, [0, 1], [len(scores) - 1], scale=1.0, split=split)
            err = (out[0].double().cpu() - want).abs() / tol
            assert (err <= 1).all(), (hi, lo, split, float(err.max()))
            assert ((lse - (2 ** 27 + math.log1p(w))).abs() <= 16).all()   # one step of fp32 there


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scores_next_to_the_largest_numbers(dim):
    """bf16 scores of 1.75 2^127 and 1.5 2^127, of either sign (times log2 e they pass fp32's range): the
    higher one takes all, wherever the two lie, and is the log-sum-exp."""
    g = gen(dim)
    page = 16
    for first, second in APART:
        n = max(first, second) + 4
        table, pages = batch_of([n - 1], [1], page, g, cols=columns(page, True))
        cache = cache_of(pages, 1, page, dim, BF16, g)
        at = torch.arange(n, device=DEV)
        where = (table[0, at // page].long(), 0, at % page)
        v = cache.v[where]
        for sign in (1, -1):
            k = torch.zeros((n, dim), device=DEV)
            k[:, 1] = 0.0 if sign > 0 else -1.75 * 2.0 ** 63   # the others are far below
            k[first, 1], k[second, 1] = (1.75 * 2.0 ** 63, 1.5 * 2.0 ** 63) if sign > 0 else (-1.5 * 2.0 ** 63, -1.75 * 2.0 ** 63)
            cache.k[where] = k.to(BF16)
            q = torch.zeros((1, 3, dim), dtype=BF16, device=DEV)
            q[..., 1] = 2.0 ** 64
            for split in (True, False):
                out, lse = attend(q, cache, table, [0, 1], [n - 1], scale=1.0, split=split)
                assert torch.equal(out, v[first].expand_as(out)), (first, second, sign, split)
                assert (lse == sign * (1.75 if sign > 0 else 1.5) * 2.0 ** 127).all()


# ---------------------------------------------------------------------------------------------
# large values

def check_relative(out, lse, want, most):
    """check_attention without the steps of fp16: weights of bf16 are right to half a step (u) of
    themselves, whatever their size, so an output is off by u + 2 ds + (most + 64) V of sum w |v| and by its
    own rounding; ds as there."""
    ref, ref_lse, size, reach = want
    u, v, dim = 2.0 ** -8, 2.0 ** -24, ref.shape[-1]
    ds = ((dim + 4) * v * reach + 4 * v * (reach + 16))[..., None]
    off = (u + 2 * ds + (most + 64) * v) * size
    tol = off + u * (ref.abs() + off)
    err = (out.double().cpu() - ref).abs() / tol
    assert (err <= 1).all(), float(err.max())
    lerr = (lse.double().cpu() - ref_lse).abs() / (ds[..., 0] + (most + 64) * v + 4 * v * (ref_lse.abs() + 16))
    assert (lerr <= 1).all(), float(lerr.max())


@pytest.mark.parametrize("kind", ["largest", "signs", "lengths", "rising", "small"])
@pytest.mark.parametrize("heads", [1, 20, 40, 100])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_bf16_values_of_every_size(dim, heads, kind):
    """Values up to the largest bf16 numbers (their sums pass fp32 before the division), alone, in all
    positions with one sign and with random ones, with lengths of 2^-40 to 2^127 in one row, behind scores
    that rise (what was summed before shrinks to nothing), and values as small as 2^-100. Contexts of one
    piece and of several, one step and many."""
    g = gen(dim + heads)
    page, top = 16, torch.finfo(BF16).max
    ctx, drafts = [0, 9, 130, 1300], [1, 2, 1, 1]
    start = [0, 1, 3, 4, 5]
    for split in (True, False):
        table, pages = batch_of(ctx, drafts, page, g, cols=columns(page, split))
        cache = cache_of(pages, 1, page, dim, BF16, g)
        v = cache.v
        if kind == "largest":
            v.fill_(top)
        elif kind == "signs":
            v.copy_(torch.where(v < 0, -top, top))
        elif kind == "lengths":
            v.copy_((v.float().sign() * torch.exp2(torch.randint(-40, 128, v.shape, device=DEV, generator=g).float())).to(BF16))
        elif kind == "small":
            v.mul_(2.0 ** -100)
        else:
            v.fill_(top)
            for b, (c, n) in enumerate(zip(ctx, drafts)):
                for p in range(c + n):
                    at = (table[b, p // page].long(), 0, p % page)
                    cache.k[at] = 0.0
                    cache.k[at][0] = 128.0 if p == c + n - 1 else float(p % 50)
                cache.v[at] = 1.0
        q = randn((5, heads, dim), BF16, g)
        if kind == "rising":
            q.zero_()
            q[..., 0] = 4.0
        out, lse = attend(q, cache, table, start, ctx, None, split=split)
        assert torch.isfinite(out).all()
        check_relative(out, lse, attention_reference(q, cache, table, start, ctx, None), 1400)


@pytest.mark.parametrize("heads", [3, 40, 100])
def test_bf16_context_values_that_are_not_finite(heads):
    """An infinity or NaN in the context reaches its own dim of all rows, and nothing else."""
    g = gen(heads)
    page, dim, ctx = 16, 128, [70, 1300]
    for split in (True, False):
        table, pages = batch_of(ctx, [1, 1], page, g, cols=columns(page, split))
        cache = cache_of(pages, 1, page, dim, BF16, g)
        q = randn((2, heads, dim), BF16, g)
        want = attention_reference(q, cache, table, [0, 1, 2], ctx, None)
        for p, d, x in ((3, 5, math.inf), (40, 77, -math.inf), (60, 100, math.nan)):
            for b in range(2):
                cache.v[table[b, p // page].long(), 0, p % page, d] = x
        out, lse = attend(q, cache, table, [0, 1, 2], ctx, None, split=split)
        assert (out[..., 5] == math.inf).all() and (out[..., 77] == -math.inf).all() and out[..., 100].isnan().all()
        out[..., [5, 77, 100]] = want[0][..., [5, 77, 100]].to(DEV).to(BF16)
        check_relative(out, lse, want, 1400)


# ---------------------------------------------------------------------------------------------
# scores that are finite where q . k or a difference of two scores is not

@pytest.mark.parametrize("heads", [1, 20, 40, 100])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=str)
def test_bf16_scores_up_to_the_largest(dtype, dim, heads):
    """A context of scores 0 with one of +1.5 2^127 and one of -1.75 2^127, whose difference passes fp32, and
    with q . k of 2^4 to 2^29 times that before the scale, in one product and as a sum of eight: the high one
    takes all; without it the zeros share, and the low one weighs nothing; alone, the low one is all there
    is. Zeros are exact, so all weights are 0, 1, or alike."""
    g = gen(dim + heads)
    page = 16
    for first, second in APART:
        n = max(first, second) + 4
        for scale in (1.0, 2.0 ** -4, 2.0 ** -29, 8.0):
            table, pages = batch_of([n - 1], [1], page, g, cols=columns(page, True))
            cache = cache_of(pages, 1, page, dim, dtype, g, scales=False)
            at = torch.arange(n, device=DEV)
            where = (table[0, at // page].long(), 0, at % page)
            k = torch.zeros((n, dim), device=DEV)
            # q . k is 3 2^126 and -3.5 2^126 over the scale, in `parts` equal products
            parts = 8 if second % 2 else 1
            size = 64.0 if dtype is E4M3 else 2.0 ** 66
            x = 2.0 ** 126 / scale / size / parts
            if x >= 2.0 ** 127:
                continue   # no bf16 query is so large
            q = torch.zeros((1, heads, dim), dtype=BF16, device=DEV)
            q[..., 3:3 + parts] = x
            for case in ("high", "low"):
                k.zero_()
                if case == "high":
                    k[first, 3:3 + parts] = 3.0 * size
                k[second, 3:3 + parts] = -3.5 * size
                assert torch.equal(k.to(dtype).float(), k)
                cache.k[where] = k.to(dtype)
                v = cache.v[where].double().cpu()
                for split in (True, False):
                    out, lse = attend(q, cache, table, [0, 1], [n - 1], scale=scale, split=split)
                    if case == "high":
                        assert torch.equal(out[0].double().cpu(), v[first].expand(heads, dim)), (first, second, scale, split)
                        assert (lse == 1.5 * 2.0 ** 127).all()
                    else:
                        rest = [p for p in range(n) if p != second]
                        want, mean = v[rest].mean(0), v[rest].abs().mean(0)
                        off = (n + 64) * 2.0 ** -24 * mean
                        assert ((out[0].double().cpu() - want).abs() <= off + 2.0 ** -8 * (want.abs() + off)).all()
                        assert ((lse.double() - math.log(n - 1)).abs() <= (n + 64) * 2.0 ** -24 + 2.0 ** -20).all()
            # a lone position
            cache.k[table[0, 0].long(), 0, 0] = k[second].to(dtype)
            out, lse = attend(q, cache, table, [0, 1], [0], scale=scale)
            assert torch.equal(out[0], cache.v[table[0, 0].long(), 0, 0].to(BF16).expand(heads, dim))
            assert (lse == -1.75 * 2.0 ** 127).all()


@pytest.mark.parametrize("scale", [2.0 ** -40, 1e-3, 0.3, 1.0, 5.0, 1e3, 2.0 ** 20])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16, E4M3], ids=str)
def test_scales_of_every_size(dtype, dim, scale):
    """Queries so large or small that scores are of ordinary size under each scale."""
    g = gen(dim)
    ctx, drafts, start = [200, 900], [3, 2], [0, 3, 5]
    for split in (True, False):
        table, pages = batch_of(ctx, drafts, 16, g, cols=columns(16, split))
        cache = cache_of(pages, 2, 16, dim, dtype, g)
        qt = F16 if dtype is F16 else BF16
        wide = dim ** -0.5 / scale
        if dtype is F16 and not 2.0 ** -10 < wide < 2.0 ** 12:
            continue
        q = (randn((5, 8, dim), torch.float32, g) * wide).to(qt)
        out, lse = attend(q, cache, table, start, ctx, None, scale=scale, split=split)
        want = attention_reference(q, cache, table, start, ctx, None, scale)
        more = 2.0 ** -22 * scale * q.float().abs().amax(-1).double().cpu() * cache.k.float().abs().sum(-1).max().item() * 1.5 \
            if dtype is E4M3 else 0.0   # bf16 queries over 8 bits: what their smallest elements may be off by
        check_attention(out, lse, want, qt, 1024, more)


# ---------------------------------------------------------------------------------------------
# the norm of large and small heads

@pytest.mark.parametrize("pairs", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.float32, BF16], ids=str)
def test_norm_of_heads_of_every_size(dtype, dim, pairs):
    """Heads whose squares pass fp32's range above and below, beside ordinary ones in the same wave."""
    g = gen(dim)
    t, heads, kv = 9, 6, 2
    q, k, v = (randn((t, n, dim), torch.float32, g) for n in (heads, kv, kv))
    for x in (q, k):
        x.clamp_(-2.9, 2.9)
        x *= torch.exp2(torch.tensor([0.0, 70, 100, 126, -70, -100, -120, 63, -40], device=DEV))[:, None, None]
        x[0, 1] *= 2.0 ** 90
        x[0, 0] *= 2.0 ** -90
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    cache = ubw.KVCache(*(torch.zeros((1, kv, 16, dim), dtype=BF16, device=DEV) for _ in "kv"))
    w = torch.rand(dim, device=DEV, generator=g) + 0.5
    freq = torch.exp2(-torch.arange(dim // 4, device=DEV).float() / 8)
    pos = slots = i32(list(range(t)))
    for eps in (0.0, 1e-6, 1e-31):
        out = ubw.qk_norm_rope(q, k, v, cache, pos, slots, freq, q_weight=w, k_weight=w, eps=eps, interleaved=pairs)
        near(out, *rope_reference(q, w, eps, pos, freq, dim // 2, pairs), BF16)
        near(cache.k[0, :, :t].transpose(0, 1), *rope_reference(k, w, eps, pos, freq, dim // 2, pairs), BF16)


@pytest.mark.parametrize("heads", [2, 20, 40, 70])
@pytest.mark.parametrize("dim", [64, 128])
def test_large_bf16_values_here_and_there(dim, heads):
    """More sequences than workgroups, every third with values up to the largest (its piece is gone through
    twice), one with an infinity: each is right whatever its workgroup did before; in a replayed graph too."""
    g = gen(heads + dim)
    seqs, page = 1600, 16
    ctx = torch.randint(0, 90, (seqs,), generator=torch.Generator().manual_seed(heads)).tolist()
    table, pages = batch_of(ctx, [1] * seqs, page, g)
    cache = cache_of(pages, 1, page, dim, BF16, g)
    for b in range(0, seqs, 3):
        rows = table[b][table[b] >= 0].long()
        cache.v[rows] = torch.where(cache.v[rows] < 0, -1.0, 1.0).to(BF16) * torch.finfo(BF16).max
    cache.v[table[7, 0].long(), 0, 0, 3] = math.inf
    q = randn((seqs, heads, dim), BF16, g)
    start = list(range(seqs + 1))
    out, lse = attend(q, cache, table, start, ctx)
    assert (out[7, :, 3] == math.inf).all()
    out[7, :, 3] = 0
    assert torch.isfinite(out).all()
    cache.v[table[7, 0].long(), 0, 0, 3] = 0
    for b in (0, 1, 2, 3, 6, 7, 8, 300, 301, 511, 512, 513, 766, 768, 769, 1023, 1024, 1025, 1300, 1536, 1598, 1599):
        want = attention_reference(q[b:b + 1], cache, table[b:b + 1], [0, 1], [ctx[b]], None)
        if b == 7:
            want[0][..., 3] = 0   # looked at above
        check_relative(out[b:b + 1], lse[b:b + 1], want, 91)
    st, cl = i32(start), i32(ctx)
    again, graph = torch.zeros_like(q), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ubw.tree_attn(q, cache, table, st, cl, max_tree=1, out=again)
    for _ in range(3):
        again.fill_(77)
        graph.replay()
        eager = ubw.tree_attn(q, cache, table, st, cl, max_tree=1)
        torch.cuda.synchronize()
        assert torch.equal(again, eager)


def test_large_bf16_values_in_some_pieces():
    """Long contexts whose pieces are gone through twice in some places, several pieces a workgroup."""
    g = gen(5)
    page, ctx, drafts, start = 256, [90000, 70000], [2, 1], [0, 2, 3]
    table, pages = batch_of(ctx, drafts, page, g)
    for heads, dim in ((8, 64), (24, 128), (320, 64)):
        cache = cache_of(pages, 8, page, dim, BF16, g)
        for p in (3, 77, 78, 200, 350):
            cache.v[table[0, p].long()] *= 2.0 ** 125
        q = randn((3, heads, dim), BF16, g)
        out, lse = attend(q, cache, table, start, ctx, split=True)
        assert torch.isfinite(out).all()
        for h in (0, heads - 1):
            hk = h // (heads // 8)
            one = ubw.KVCache(cache.k[:, hk:hk + 1].contiguous(), cache.v[:, hk:hk + 1].contiguous())
            want = attention_reference(q[:, h:h + 1].contiguous(), one, table, start, ctx, None)
            check_relative(out[:, h:h + 1], lse[:, h:h + 1], want, 90002)
