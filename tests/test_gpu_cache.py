"""GPU parity of the key/value cache calls with plain 64-bit definitions on the host's side: norm and
rotation into a paged cache, attention of trees of tokens over it, and the cache's pages.

Tolerances count roundings: u = finfo(type).eps / 2 is half a step of a type, v = 2^-24 that of fp32.
Whole numbers and moved bytes are compared exactly.
"""
import math

import numpy as np
import pytest

import oracle
import ultra_bit_weight_uint32_amd as ubw
from workloads import make_gemv

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, E4M3, F32, F64 = torch.float16, torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.float64
V = 2.0 ** -24


def half_step(dtype):
    return 2.0 ** -4 if dtype is E4M3 else torch.finfo(dtype).eps / 2


def smallest(dtype):   # half the spacing next to zero
    return {F16: 2.0 ** -25, BF16: 2.0 ** -134, E4M3: 2.0 ** -10}[dtype]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(shape, dtype, g):
    x = torch.randn(shape, device=DEV, generator=g)
    return x.clamp(-440, 440).to(dtype) if dtype is E4M3 else x.to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def cache_of(pages, heads, page, dim, dtype, g, token_major=False, scales=True):
    """A cache of normal values; token_major: [pages, page, heads, dim] seen as [pages, heads, page, dim]."""
    shape = (pages, page, heads, dim) if token_major else (pages, heads, page, dim)
    k, v = randn(shape, dtype, g), randn(shape, dtype, g)
    if token_major:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    ks = vs = None
    if dtype is E4M3 and scales:
        ks, vs = (torch.rand(heads, device=DEV, generator=g) + 0.5 for _ in "kv")
    return ubw.KVCache(k, v, ks, vs)


# ---------------------------------------------------------------------------------------------
# norm, rotation, store

ROPE = [  # tokens, heads, kv, dim, source, cache, out, rot, interleaved, norm, page
    (1, 64, 8, 128, F32, F16, F16, 128, False, False, 16), (1, 1, 1, 64, F16, F16, F16, 64, True, True, 16),
    (3, 12, 4, 64, BF16, BF16, BF16, 32, False, True, 32), (17, 5, 5, 128, F32, BF16, BF16, 96, False, True, 16),
    (7, 8, 2, 256, F16, F16, BF16, 256, False, True, 64), (9, 3, 1, 256, F32, E4M3, F16, 70, True, False, 16),
    (40, 7, 7, 128, BF16, E4M3, BF16, 64, False, True, 128), (5, 16, 1, 64, F32, E4M3, F16, 2, True, True, 16),
    (2, 40, 8, 128, F16, F16, F16, 0, False, True, 16), (700, 32, 32, 128, F32, F16, F16, 128, True, True, 16),
    (33, 2, 2, 128, F16, BF16, F16, 6, True, True, 1024), (2100, 2, 1, 64, BF16, BF16, BF16, 64, False, False, 16),
]


def rope_reference(x, w, eps, positions, freq, rot, pairs):
    """(y of the definition in 64 bits, the size of the two terms each element adds)."""
    x = x.double().cpu()
    if w is not None:
        x = x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * w.double().cpu()
    y, size = x.clone(), x.abs()
    if rot:
        t = positions.double().cpu()[:, None, None] * freq.double().cpu()
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
        y[..., a] = x[..., a] * t.cos() - x[..., b] * t.sin()
        y[..., b] = x[..., b] * t.cos() + x[..., a] * t.sin()
        size = size.clone()
        size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, size


def near(got, want, size, dtype, scale=None):
    """Rounded once to `dtype` from fp32 arithmetic: the norm is a sum of head_dim squares in 16 lanes
    (at most 16 + 4 roundings), a square root, a division and two products (under 30 in all), cosine and
    sine come from an angle reduced in 64 bits and rounded to 2^-26 of a turn (under 4 roundings of size
    V), two products and a sum: under 40 V of the terms' size. An 8-bit value is divided by its scale
    first (one rounding more)."""
    off = 40 * V * size
    s = torch.ones(()) if scale is None else scale.double().cpu()[:, None]
    big = 448.0 if dtype is E4M3 else math.inf
    ref = (want / s).clamp(-big, big)
    tol = half_step(dtype) * (ref.abs() + off / s) + off / s + V * ref.abs() + smallest(dtype)
    got = got.double().cpu()
    bad = (got - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got - ref).abs() / tol).max()))


@pytest.mark.parametrize("case", ROPE, ids=str)
def test_rope(case):
    t, h, kv, dim, src, ct, ot, rot, pairs, norm, page = case
    g = gen(sum(map(int, (t, h, kv, dim, rot))))
    fused = randn((t, (h + 2 * kv) * dim), src, g)
    q, k, v = (x.unflatten(1, (-1, dim)) for x in fused.split([h * dim, kv * dim, kv * dim], 1))
    pages = -(-t // page) + 2
    cache = cache_of(pages, kv, page, dim, ct, g, token_major=t % 2 == 1)
    cache.k.zero_(), cache.v.zero_()
    pos = torch.randint(0, 1 << 20, (t,), dtype=torch.int32, device=DEV, generator=g)
    pos[0] = 2147483647
    slots = torch.randperm(pages * page, device=DEV, generator=g)[:t].to(torch.int32)
    if t > 2:
        slots[1], slots[2] = -1, pages * page   # padding: not stored
    freq = (10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=F64) / max(rot, 1))).to(F32) if rot else None
    qw, kw = (torch.rand(dim, device=DEV, generator=g) + 0.5 if norm else None for _ in "qk")
    got = ubw.qk_norm_rope(q, k, v, cache, pos, slots, freq, q_weight=qw, k_weight=kw, eps=1e-5, interleaved=pairs,
                           out_dtype=ot)
    assert got.dtype is ot and got.shape == (t, h, dim)
    near(got, *rope_reference(q, qw, 1e-5, pos, freq, rot, pairs), ot)
    kr, ksize = rope_reference(k, kw, 1e-5, pos, freq, rot, pairs)
    at = slots.long().cpu()
    ok = (at >= 0) & (at < pages * page)
    for c, want, size, scale in ((cache.k, kr, ksize, cache.k_scale), (cache.v, v.double().cpu(), 0 * ksize, cache.v_scale)):
        flat = c.float().cpu().transpose(1, 2).reshape(-1, kv, dim)   # [slot, head, dim]
        near(flat[at[ok]], want[ok], size[ok], ct, scale)
        rest = torch.ones(pages * page, dtype=torch.bool)
        rest[at[ok]] = False
        assert not flat[rest].any()


def test_rope_of_unusual_values():
    """8 bits: what is too large becomes the largest value, NaN stays; a head of zeros with eps 0 is NaN in
    itself alone; infinities rotate as the formula has it and leave the dims behind rot alone."""
    dim = 64
    q, k, v = (torch.ones((2, 1, dim), device=DEV) for _ in "qkv")
    v[0, 0, :4] = torch.tensor([1e6, -math.inf, math.nan, 449.0])
    k[0, 0, 40] = math.inf
    q[1] = 0
    cache = ubw.KVCache(*(torch.zeros((1, 1, 16, dim), device=DEV, dtype=E4M3) for _ in "kv"))
    w = torch.ones(dim, device=DEV)
    out = ubw.qk_norm_rope(q, k, v, cache, i32([0, 5]), i32([3, 9]), torch.ones(16, device=DEV), q_weight=w, eps=0.0)
    assert cache.v[0, 0, 3, :5].float().tolist()[:2] == [448, -448] and cache.v[0, 0, 3, 2].float().isnan()
    assert cache.v[0, 0, 3, 3:5].float().tolist() == [448, 1]
    assert cache.k[0, 0, 3, 40].float() == 448 and (cache.k[0, 0, 3, 32:40].float() == 1).all()
    assert out[1].isnan().all() and (out[0] == 1).all()


def test_rope_far_rows_of_a_large_cache():
    """Pages whose byte offsets pass 32 bits."""
    dim, page, pages = 256, 1024, 9000   # 4.7 GB each
    k, v = (torch.empty((pages, 1, page, dim), dtype=F16, device=DEV) for _ in "kv")
    k[-1] = 0
    v[-1] = 0
    cache = ubw.KVCache(k, v)
    g = gen(3)
    x = randn((2, 1, dim), F16, g)
    slot = pages * page - 7
    ubw.qk_norm_rope(x, x, x, cache, i32([0, 0]), i32([slot, -1]), None)
    assert torch.equal(k[-1, 0, page - 7], x[0, 0]) and torch.equal(v[-1, 0, page - 7], x[0, 0])
    assert int((k[-1] != 0).any(-1).sum()) == 1
    # attention over it, and moving its pages
    table = i32([[pages - 1]])
    k[-1, 0], v[-1, 0] = randn((page, dim), F16, g), randn((page, dim), F16, g)
    out, lse, want = attend_and_check(x[:1].contiguous(), cache, table, [0, 1], [999], None)
    k[0, 0], v[0, 0] = 0, 0
    ubw.cache_copy_pages(cache, i32([[pages - 1, 0]]))
    assert torch.equal(k[0], k[-1]) and torch.equal(v[0], v[-1])
    was = k[-1, 0, 505].clone()
    ubw.cache_compact(cache, table, i32([500]), i32([[5]]))
    assert torch.equal(k[-1, 0, 500], was)


# ---------------------------------------------------------------------------------------------
# attention

def seen_of(ctx, n, masks, row0, positions):
    """[n, positions] truth: what each token of a sequence sees."""
    at = torch.arange(positions)
    out = torch.zeros((n, positions), dtype=torch.bool)
    for i in range(n):
        bits = (1 << (i + 1)) - 1 if masks is None else int(masks[row0 + i])
        d = at - ctx
        tree = torch.tensor([(0 <= int(x) < min(n, 64)) and bool((bits >> int(x)) & 1) for x in d])
        out[i] = (d < 0) | tree
    return out


def attention_reference(q, cache, table, start, ctx, masks, scale=None):
    """out, lse in 64 bits; and of each output sum w |v|, of each row the largest scale sum |q||k| and the
    positions there are."""
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
    table = table.cpu()
    masks = None if masks is None else [int(m) & (2 ** 64 - 1) for m in masks.tolist()]
    for b, c in enumerate(ctx):
        n = start[b + 1] - start[b]
        if n == 0:
            continue
        length = min(max(c, 0) + n, table.shape[1] * page)
        pg = table[b, (torch.arange(length) // page)].long()
        valid = (pg >= 0) & (pg < cache.pages)
        sees = seen_of(max(c, 0), n, masks, start[b], length) & valid
        rows = torch.arange(length) % page
        for h in range(heads):
            hk = h // (heads // kv)
            kk, vv = k[pg.clamp(0, cache.pages - 1), hk, rows], v[pg.clamp(0, cache.pages - 1), hk, rows]
            for i in range(n):
                on = sees[i]
                if not on.any():
                    continue
                x = q[start[b] + i, h]
                s = scale * (kk[on] @ x)
                r = start[b] + i
                lse[r, h] = torch.logsumexp(s, 0)
                w = torch.softmax(s, 0)
                out[r, h] = w @ vv[on]
                size[r, h] = w @ vv[on].abs()
                reach[r, h] = scale * (kk[on].abs() @ x.abs()).max()
    return out, lse, size, reach


def attend_and_check(q, cache, table, start, ctx, masks, scale=None, split=True, **kw):
    t, heads, dim = q.shape
    tree = max(b - a for a, b in zip(start, start[1:]))
    ws = ubw.tree_attn_workspace(len(ctx), max(tree, 1), heads, cache.kv_heads, dim, DEV) if split else None
    if ws is not None:
        ws.fill_(math.nan)   # scratch: what it held does not matter
    out = torch.full((t, heads, dim), 77.0, dtype=q.dtype, device=DEV)
    lse = torch.full((t, heads), 77.0, device=DEV)
    ubw.tree_attn(q, cache, table, i32(start), i32(ctx), masks, max_tree=max(tree, 1), scale=scale, out=out, lse=lse,
                  workspace=ws, **kw)
    want = attention_reference(q, cache, table, start, ctx, masks, scale)
    check_attention(out, lse, want, q.dtype, table.shape[1] * cache.page_size)
    return out, lse, want


def check_attention(out, lse, want, dtype, most, more=0.0):
    """Against 64 bits. Scores: a sum of dim products of exact factors and a product with the scale, then
    the difference to the maximum before the exponential (which is good to 2 V): ds <= (dim + 4) V reach
    + 4 V (|s| + 16) with |s| <= reach. Weights are off by 2 ds relatively, each rounded to the type
    once (u), or by half of fp16's smallest step, 2^-25 where the largest weight is 2^7 or more. Sums
    over `most` positions, the parts' scaling and the division: (most + 64) V. Then one rounding. `more`:
    what scores are off by besides."""
    ref, ref_lse, size, reach = want
    dim = ref.shape[-1]
    u = half_step(dtype)
    ds = ((dim + 4) * V * reach + 4 * V * (reach + 16) + more)[..., None]
    rel = u + 2 * ds + (most + 64) * V
    # the smallest steps add at most most 2^-32 of the largest |v| < 6 (normal values, scales below 1.5)
    off = rel * size + most * 2.0 ** -32 * 9
    tol = off + u * (ref.abs() + off) + smallest(dtype)
    got = out.double().cpu()
    rows = torch.isfinite(ref_lse)
    assert torch.equal(lse.cpu()[~rows], torch.full_like(lse.cpu()[~rows], -math.inf))
    assert not got[~rows].any()
    err = (got - ref).abs() / tol
    assert (err[rows] <= 1).all(), float(err[rows].max())
    ltol = ds[..., 0] + (most + 64) * V + 4 * V * (ref_lse.abs() + 16)
    lerr = (lse.double().cpu() - ref_lse).abs() / ltol
    assert (lerr[rows] <= 1).all(), float(lerr[rows].max())


def batch_of(ctx, drafts, page, g, spare=2, cols=0):
    """(table, pages): pages in random order, -1 behind what a sequence needs."""
    need = [-(-(c + n) // page) for c, n in zip(ctx, drafts)]
    pages = sum(need) + spare
    order = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)
    table = torch.full((len(ctx), max(max(need), cols, 1)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


ATTEND = [  # heads, kv, dim, q type, cache type, page, contexts, tokens, masks
    (1, 1, 64, F16, F16, 16, [0], [1], "none"), (8, 8, 128, F16, F16, 16, [37], [1], "none"),
    (8, 1, 128, BF16, BF16, 16, [1, 15, 16, 17, 31, 32, 33, 127], [1] * 8, "none"),
    (6, 2, 128, F16, F16, 32, [128, 129, 0, 511, 5], [1, 3, 2, 1, 0], "random"),
    (16, 2, 64, BF16, BF16, 64, [100, 0, 257], [5, 16, 33], "random"),
    (8, 1, 128, F16, F16, 16, [300, 64], [16, 7], "none"), (4, 2, 128, BF16, BF16, 128, [61, 0], [64, 64], "random"),
    (5, 5, 256, F16, F16, 16, [97, 12], [3, 17], "random"), (16, 1, 256, BF16, BF16, 64, [200], [5], "none"),
    (8, 8, 64, F16, E4M3, 16, [63, 64, 65], [1, 1, 1], "none"), (12, 4, 128, BF16, E4M3, 32, [250, 31], [9, 2], "random"),
    (8, 1, 256, F16, E4M3, 16, [130], [6], "random"), (8, 2, 128, F16, E4M3, 1024, [1500, 3], [20, 64], "random"),
    (3, 1, 128, BF16, BF16, 16, [1000, 2, 640], [2, 40, 11], "random"), (64, 8, 128, F16, F16, 16, [700], [1], "none"),
    (16, 16, 64, BF16, E4M3, 16, [40], [31], "none"),
    # several row blocks over the same keys and values
    (16, 1, 128, BF16, BF16, 16, [513, 77], [33, 20], "random"), (24, 2, 64, F16, F16, 16, [400], [50], "random"),
    (8, 1, 64, F16, E4M3, 32, [300, 0], [40, 64], "random"), (7, 1, 256, BF16, E4M3, 16, [260], [30], "none"),
    # more pieces of a row than its four waves take at once
    (2, 1, 64, F16, F16, 256, [60000], [1], "none"),
]


@pytest.mark.parametrize("split", [True, False, "long table"])
@pytest.mark.parametrize("case", ATTEND, ids=str)
def test_attention(case, split):
    """With a workspace, without one, and with a table so long that short contexts are split too."""
    heads, kv, dim, qt, ct, page, ctx, drafts, masks = case
    g = gen(heads + dim + page + sum(ctx))
    table, pages = batch_of(ctx, drafts, page, g, cols=1 + 1024 // page if split == "long table" else 0)
    cache = cache_of(pages, kv, page, dim, ct, g, token_major=heads % 2 == 1)
    t = sum(drafts)
    start = [0] + list(np.cumsum(drafts))
    q = randn((t + 3, heads + 2, dim), qt, g)[:t, 1:-1] if heads % 4 == 0 else randn((t, heads, dim), qt, g)
    m = None
    if masks == "random":
        m = torch.randint(-2 ** 63, 2 ** 63 - 1, (t,), device=DEV, generator=g)
        m[torch.rand(t, device=DEV, generator=g) < 0.2] = 0
        m[-1] = -1
    out, lse, _ = attend_and_check(q, cache, table, start, ctx, m, split=split)
    # the same call again gives the same bits, and a stated length changes nothing but the split
    again = attend_and_check(q, cache, table, start, ctx, m, split=split, max_len=max(c + n for c, n in zip(ctx, drafts)))
    assert split or (torch.equal(out, again[0]) and torch.equal(lse, again[1]))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("tokens", [1, 4, 8, 33])
def test_attention_of_queries_of_many_sizes(tokens, dim):
    """bf16 queries whose elements lie far apart, over 8-bit keys. Elements may be taken to 2^-22 of the
    row's largest: scores are off by up to 2^-22 max |q| scale sum |k| more. Among the rows are zeros, one
    element alone, the smallest numbers, and one large element among small ones."""
    g = gen(90 + dim + tokens)
    ctx = [150]
    table, pages = batch_of(ctx, [tokens], 16, g)
    cache = cache_of(pages, 1, 16, dim, E4M3, g)
    q = randn((tokens, 8, dim), F32, g)
    q *= torch.exp2(torch.randint(-20, 2, q.shape, device=DEV, generator=g).float())
    q[:, 1] = 0
    q[:, 2, 1:] = 0
    q[:, 3] *= 2.0 ** -100
    q[:, 4] *= 2.0 ** -122   # to the smallest bf16 numbers and below
    q[:, 5, dim - 1] = 3.0
    q[:, 6, 5] = 2.0 ** 20
    q = q.to(BF16)
    out = torch.empty_like(q)
    lse = torch.empty((tokens, 8), device=DEV)
    start = [0, tokens]
    ubw.tree_attn(q, cache, table, i32(start), i32(ctx), None, max_tree=tokens, out=out, lse=lse)
    want = attention_reference(q, cache, table, start, ctx, None)
    k = cache.k.float().abs().sum(-1).max().item() * (1.0 if cache.k_scale is None else cache.k_scale.max().item())
    more = 2.0 ** -22 * dim ** -0.5 * k * q.float().abs().amax(-1).double().cpu()
    check_attention(out, lse, want, BF16, table.shape[1] * cache.page_size, more)


def test_attention_repeats_bit_for_bit():
    g = gen(5)
    ctx, drafts = [3000, 20, 1111], [4, 1, 16]
    table, pages = batch_of(ctx, drafts, 16, g)
    cache = cache_of(pages, 2, 16, 128, BF16, g)
    q = randn((21, 16, 128), BF16, g)
    ws = ubw.tree_attn_workspace(3, 16, 16, 2, 128, DEV)
    args = (q, cache, table, i32([0, 4, 5, 21]), i32(ctx))
    first = ubw.tree_attn(*args, max_tree=16, workspace=ws)
    for _ in range(5):
        assert torch.equal(first, ubw.tree_attn(*args, max_tree=16, workspace=ws))


@pytest.mark.parametrize("dtype", [F16, BF16, E4M3])
@pytest.mark.parametrize("split", [True, False])
def test_attention_ignores_what_is_not_seen(dtype, split):
    """NaN and infinities behind a sequence's end, in unseen tree tokens, and in the pages of others reach
    nothing; the outputs are those of a cache with zeros there."""
    heads, kv, dim, page = 8, 2, 128, 32
    ctx, drafts = [70, 0, 131], [6, 5, 9]
    g = gen(11)
    table, pages = batch_of(ctx, drafts, page, g)
    cache = cache_of(pages, kv, page, dim, dtype, g)
    qt = F16 if dtype is E4M3 else dtype
    q = randn((20, heads, dim), qt, g)
    start = [0, 6, 11, 20]
    masks = torch.randint(0, 2 ** 40, (20,), device=DEV, generator=g)
    hidden = {0: 2, 1: 0, 2: 7}   # this tree token is seen by no one
    for b, j in hidden.items():
        masks[start[b]:start[b + 1]] &= ~(1 << j)
    masks[12] = 0                 # sees its context alone
    masks[7] = 0                  # and nothing
    want = attend_and_check(q, cache, table, start, ctx, masks, split=split)
    spoiled = torch.zeros((pages, page), dtype=torch.bool, device=DEV)
    spoiled[:] = True
    for b, (c, n) in enumerate(zip(ctx, drafts)):
        for p in range(c + n):
            if p - c != hidden[b]:
                spoiled[table[b, p // page].long(), p % page] = False
    bad = spoiled[:, None, :, None].expand(cache.k.shape)
    for x, val in ((cache.k, math.nan), (cache.v, math.nan)) if dtype is E4M3 else ((cache.k, math.inf), (cache.v, -math.inf)):
        x.copy_(torch.where(bad, torch.full_like(x.float(), val), x.float()).to(dtype))
    ws = ubw.tree_attn_workspace(3, 9, heads, kv, dim, DEV) if split else None
    lse = torch.empty((20, heads), device=DEV)
    out = ubw.tree_attn(q, cache, table, i32(start), i32(ctx), masks, max_tree=9, lse=lse, workspace=ws)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    cache.v.copy_(torch.where(bad, torch.full_like(cache.v.float(), math.nan), cache.v.float()).to(dtype))
    assert torch.equal(ubw.tree_attn(q, cache, table, i32(start), i32(ctx), masks, max_tree=9, workspace=ws), want[0])


@pytest.mark.parametrize("dtype", [F16, E4M3])
def test_a_tree_token_that_is_not_finite_reaches_those_who_see_it(dtype):
    heads, kv, dim, page = 4, 2, 64, 16
    g = gen(12)
    table, pages = batch_of([21], [4], page, g)
    cache = cache_of(pages, kv, page, dim, dtype, g, scales=False)
    q = randn((4, heads, dim), F16, g)
    masks = torch.tensor([1, 3, 5, 13], device=DEV)   # token 1 is seen by itself alone
    clean = ubw.tree_attn(q, cache, table, i32([0, 4]), i32([21]), masks, max_tree=4)
    cache.v[table[0, 22 // page].long(), 1, 22 % page, 5] = math.nan
    got = ubw.tree_attn(q, cache, table, i32([0, 4]), i32([21]), masks, max_tree=4)
    nan = torch.zeros_like(got, dtype=torch.bool)
    nan[1, 2:, 5] = True
    assert torch.equal(got.isnan(), nan)
    assert torch.equal(got[~nan], clean[~nan])


def test_attention_of_infinite_scores():
    """A row with a score of +inf is NaN, as its softmax; its neighbours are untouched. Scores of -inf
    weigh nothing."""
    g = gen(13)
    table, pages = batch_of([40], [2], 16, g)
    cache = cache_of(pages, 1, 16, 64, F16, g)
    q = randn((2, 2, 64), F16, g).abs()
    clean = ubw.tree_attn(q, cache, table, i32([0, 2]), i32([40]), max_tree=2)
    spot = table[0, 0].long()
    was = cache.k[spot, 0, 3, 7].clone()
    cache.k[spot, 0, 3, 7] = math.inf
    assert ubw.tree_attn(q, cache, table, i32([0, 2]), i32([40]), max_tree=2).isnan().all()
    cache.k[spot, 0, 3, 7] = -math.inf
    got = ubw.tree_attn(q, cache, table, i32([0, 2]), i32([40]), max_tree=2)
    assert torch.isfinite(got).all() and not torch.equal(got, clean)
    cache.k[spot, 0, 3, 7] = was
    assert torch.equal(ubw.tree_attn(q, cache, table, i32([0, 2]), i32([40]), max_tree=2), clean)


def test_attention_scores_of_every_size():
    """Scores that grow along the context (the maximum moves all the time), shrink, and lie far apart."""
    heads, dim, page, n = 2, 64, 16, 700
    g = gen(14)
    table, pages = batch_of([n], [1], page, g)
    for kind in range(4):
        cache = cache_of(pages, 1, page, dim, F16, g)
        q = torch.zeros((1, heads, dim), dtype=F16, device=DEV)
        q[..., 0] = 1
        ramp = torch.arange(n + 1, device=DEV) * [0.7, -0.7, 0.0, 30.0][kind]
        ramp = ramp % 60000 if kind == 3 else ramp
        for p in range(n + 1):
            cache.k[table[0, p // page].long(), 0, p % page, 0] = ramp[p].to(F16)
        for split in (True, False):
            attend_and_check(q, cache, table, [0, 1], [n], None, scale=1.0, split=split)


def test_attention_of_scores_near_the_lowest_number():
    """A lone position weighs 1 however low its score is, and of two far ones the higher takes all."""
    cache = cache_of(1, 1, 16, 64, BF16, gen(18))
    cache.k.zero_()
    q = torch.zeros((2, 2, 64), dtype=BF16, device=DEV)
    q[..., 0] = 1e19
    cache.k[0, 0, :2, 0] = torch.tensor([-1e19, -2e19], device=DEV)
    table = i32([[0]])
    for split in (True, False):
        ws = ubw.tree_attn_workspace(1, 2, 2, 1, 64, DEV) if split else None
        lse = torch.empty((2, 2), device=DEV)
        out = ubw.tree_attn(q, cache, table, i32([0, 2]), i32([0]), max_tree=2, scale=1.0, lse=lse, workspace=ws)
        assert torch.equal(out, cache.v[0, 0, 0].expand_as(out))
        assert torch.allclose(lse, torch.full_like(lse, float(q[0, 0, 0].double() * cache.k[0, 0, 0, 0].double())), rtol=1e-6)


def test_attention_of_one_layer_of_many():
    g = gen(19)
    k, v = (randn((3, 5, 2, 16, 64), BF16, g) for _ in "kv")
    cache = ubw.KVCache(k, v)
    q, table = randn((2, 4, 64), BF16, g), i32([[4, 2, 0, 1]])
    for layer in range(3):
        attend_and_check(q, cache.layer(layer), table, [0, 2], [50], None)
    # a call that takes one layer takes the first of many
    first = ubw.tree_attn(q, cache, table, i32([0, 2]), i32([50]), max_tree=2)
    assert torch.equal(first, ubw.tree_attn(q, cache.layer(0), table, i32([0, 2]), i32([50]), max_tree=2))


def test_attention_cuts_what_it_cannot_use():
    """Lengths beyond the table, entries that are no pages, negative contexts, rows of no sequence, trees
    over max_tree: cut as documented, the rest right, nothing else written."""
    heads, kv, dim, page = 4, 2, 64, 16
    g = gen(15)
    cache = cache_of(9, kv, page, dim, F16, g)
    table = i32([[3, 99, 5], [1, 2, -7], [0, 4, 6]])
    ctx, start = [30, 100, -5], [0, 2, 4, 7]
    q = randn((9, heads, dim), F16, g)
    for split in (True, False):
        out, lse = torch.full_like(q, 77), torch.full((9, heads), 77.0, device=DEV)
        ws = ubw.tree_attn_workspace(3, 3, heads, kv, dim, DEV) if split else None
        ubw.tree_attn(q, cache, table, i32(start), i32(ctx), max_tree=3, out=out, lse=lse, workspace=ws)
        want = attention_reference(q[:7], cache, table, start, ctx, None)
        check_attention(out[:7], lse[:7], want, F16, 48)
        assert (out[7:] == 77).all() and (lse[7:] == 77).all()
        out.fill_(77)
        ubw.tree_attn(q, cache, table, i32(start), i32(ctx), max_tree=2, out=out, workspace=None)
        assert (out[6:] == 77).all() and not (out[5] == 77).any()   # the third token of the last tree
        # starts that do not ascend, or pass the rows there are: nothing outside is touched
        out.fill_(77)
        ubw.tree_attn(q[:7], cache, table, i32([5, -3, 1000, 2]), i32([2 ** 31 - 1, 0, -2 ** 31]), max_tree=3, out=out[:7],
                      workspace=ws)
        assert (out[7:] == 77).all()
    empty = ubw.tree_attn(q[:0], cache, table, i32([0, 0, 0, 0]), i32(ctx), max_tree=1)
    assert empty.shape == (0, heads, dim)


def test_attention_batches_larger_than_a_workgroup():
    g = gen(16)
    r = np.random.default_rng(16)
    ctx, drafts = r.integers(0, 60, 700).tolist(), r.integers(0, 3, 700).tolist()
    table, pages = batch_of(ctx, drafts, 16, g)
    cache = cache_of(pages, 1, 16, 64, BF16, g)
    q = randn((sum(drafts), 1, 64), BF16, g)
    start = [0] + list(np.cumsum(drafts))
    for split in (True, False):
        attend_and_check(q, cache, table, start, ctx, None, split=split)


def test_attention_on_other_streams_and_in_graphs():
    """Two streams with workspaces of their own at once, and a captured call replayed between eager ones,
    its lengths changed in place."""
    heads, kv, dim, page = 16, 2, 128, 16
    g = gen(17)
    table, pages = batch_of([2000, 900], [4, 4], page, g)
    cache = cache_of(pages, kv, page, dim, F16, g)
    qs = [randn((8, heads, dim), F16, g) for _ in range(2)]
    start, ctx = i32([0, 4, 8]), i32([2000, 900])
    wss = [ubw.tree_attn_workspace(2, 4, heads, kv, dim, DEV) for _ in range(2)]
    want = [ubw.tree_attn(q, cache, table, start, ctx, max_tree=4, workspace=wss[0]) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [torch.empty_like(q) for q in qs]
    for _ in range(10):
        for s, q, o, ws in zip(streams, qs, got, wss):
            with torch.cuda.stream(s):
                ubw.tree_attn(q, cache, table, start, ctx, max_tree=4, out=o, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

    graph, out = torch.cuda.CUDAGraph(), torch.zeros_like(qs[0])
    q = qs[0].clone()
    with torch.cuda.graph(graph):
        ubw.tree_attn(q, cache, table, start, ctx, max_tree=4, out=out, workspace=wss[1])
    for step, lens in enumerate(([2000, 900], [3, 1], [0, 800], [1999, 64], [2000, 900])):
        ctx.copy_(i32(lens))
        q.copy_(qs[step % 2])
        out.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ubw.tree_attn(q, cache, table, start, ctx, max_tree=4, workspace=wss[0])), step


# ---------------------------------------------------------------------------------------------
# pages

def bits(x):
    return x.view(torch.uint8 if x.dtype is E4M3 else torch.int16)


@pytest.mark.parametrize("dtype,layers,kv,page,dim,token_major",
                         [(F16, 1, 1, 16, 64, False), (BF16, 3, 5, 32, 128, False), (E4M3, 2, 8, 16, 64, True),
                          (F16, 2, 3, 128, 256, True), (E4M3, 5, 1, 1024, 256, False)])
def test_copy_pages(dtype, layers, kv, page, dim, token_major):
    g = gen(page + dim)
    pages = 23
    shape = (layers, pages, page, kv, dim) if token_major else (layers, pages, kv, page, dim)
    k, v = randn(shape, dtype, g), randn(shape, dtype, g)
    if token_major:
        k, v = k.transpose(2, 3), v.transpose(2, 3)
    cache = ubw.KVCache(k, v)
    pairs = [[0, 7], [22, 1], [0, 2], [-1, -1], [5, 23], [-4, 3], [30, 4], [9, 9], [21, 20]]
    want = []
    for x in (k, v):
        w = bits(x).clone()
        for a, b in pairs:
            if 0 <= a < pages and 0 <= b < pages:
                w[:, b] = bits(x)[:, a]
        want.append(w)
    ubw.cache_copy_pages(cache, i32(pairs))
    assert torch.equal(bits(k), want[0]) and torch.equal(bits(v), want[1])
    ubw.cache_copy_pages(cache, i32([]).view(0, 2))
    one = cache.layer(layers - 1)
    ubw.cache_copy_pages(one, i32([[2, 11]]))
    want[0][-1, 11] = want[0][-1, 2]
    assert torch.equal(bits(k), want[0])


def compact_model(x, table, page, ctx, keep):
    w = bits(x).clone()
    pages = x.shape[1]
    for b, c in enumerate(ctx):
        last = -1
        for i, j in enumerate(keep[b]):
            if c < 0 or j <= last:
                break
            last = j
            at = [divmod(c + p, page) for p in (j, i)]
            if any(col >= table.shape[1] or not 0 <= int(table[b, col]) < pages for col, _ in at):
                continue
            w[:, int(table[b, at[1][0]]), :, at[1][1]] = w[:, int(table[b, at[0][0]]), :, at[0][1]].clone()
    return w


@pytest.mark.parametrize("dtype,layers,kv,page,dim", [(F16, 1, 1, 16, 64), (BF16, 3, 5, 32, 128), (E4M3, 2, 8, 16, 64),
                                                      (F16, 2, 3, 16, 256)])
def test_compact(dtype, layers, kv, page, dim):
    g = gen(page + dim + 1)
    r = np.random.default_rng(dim)
    ctx, drafts = [0, 1, 15, 16, 17, 100, 63, 3], [64] * 8
    table, pages = batch_of(ctx, drafts, page, g)
    k, v = (randn((layers, pages, kv, page, dim), dtype, g) for _ in "kv")
    cache = ubw.KVCache(k, v)
    width = 40
    keep = []
    for b in range(8):
        m = [0, 1, 8, 9, 16, 40, 25, 33][b]
        keep.append(sorted(r.choice(64, m, replace=False).tolist()) + [-1] * (width - m))
    keep[6][3] = keep[6][2]          # a list ends where it does not ascend
    keep[7][10] = 0
    keep[4] = list(range(40))        # already in place
    for _ in range(2):               # twice: lists of a second round move what the first one left
        want = [compact_model(x, table, page, ctx, keep) for x in (k, v)]
        ubw.cache_compact(cache, table, i32(ctx), i32(keep))
        assert torch.equal(bits(k), want[0]) and torch.equal(bits(v), want[1])
    bad = table.clone()
    bad[0, 0], bad[1, 1], bad[2, :] = -1, pages, 2 ** 31 - 1
    rows = torch.nn.functional.pad(bad, (0, 3))[:, :bad.shape[1] - 1]   # fewer columns, rows apart
    lens = list(ctx)
    lens[3], lens[5] = -16, 2 ** 31 - 1
    want = [compact_model(x, rows, page, lens, keep) for x in (k, v)]
    ubw.cache_compact(cache, rows, i32(lens), i32(keep))
    assert torch.equal(bits(k), want[0]) and torch.equal(bits(v), want[1])


class PoolModel:
    """The pool's calls one sequence after the other."""

    def __init__(self, pages, page, seqs, cols):
        self.ref, self.page, self.cols = [0] * pages, page, cols
        self.rows, self.len, self.status = [[] for _ in range(seqs)], [0] * seqs, 0

    def trim(self, new):
        for s, n in enumerate(new):
            if n < 0:
                continue
            cut = -(-n // self.page)
            if cut > len(self.rows[s]):
                self.status |= 2
                continue
            for p in self.rows[s][cut:]:
                self.ref[p] -= 1
            self.rows[s], self.len[s] = self.rows[s][:cut], n

    def fork(self, parents):
        was = [list(r) for r in self.rows]
        for s, p in enumerate(parents):
            if p < 0:
                continue
            if p >= len(parents) or p == s or parents[p] >= 0 or was[s]:
                self.status |= 2
                continue
            n = -(-self.len[p] // self.page)
            self.rows[s], self.len[s] = was[p][:n], self.len[p]
            for q in self.rows[s]:
                self.ref[q] += 1

    def reserve(self, room):
        pairs = [[-1, -1] for _ in room]
        need = []
        for s, r in enumerate(room):
            want = -(-(self.len[s] + r) // self.page)
            if r <= 0 or want > self.cols:
                self.status |= 2 if r > 0 else 0
                need.append((0, None))
                continue
            at = self.len[s] // self.page
            own = at < len(self.rows[s]) and self.ref[self.rows[s][at]] > 1
            need.append((max(0, want - len(self.rows[s])), at if own else None))
        free = [p for p, n in enumerate(self.ref) if n == 0]
        if sum(n + (at is not None) for n, at in need) > len(free):
            self.status |= 1
            return pairs
        old = []
        for s, (n, at) in enumerate(need):
            if at is not None:
                pairs[s] = [self.rows[s][at], free.pop(0)]
                old.append(pairs[s][0])
                self.rows[s][at] = pairs[s][1]
                self.ref[pairs[s][1]] = 1
            for _ in range(n):
                self.rows[s].append(free.pop(0))
                self.ref[self.rows[s][-1]] = 1
        for p in old:
            self.ref[p] -= 1
        return pairs

    def check(self, pool):
        assert pool.status.item() == self.status
        assert pool.len.tolist() == self.len
        assert pool.held.tolist() == [len(r) for r in self.rows]
        assert pool.table.tolist() == [r + [-1] * (self.cols - len(r)) for r in self.rows]
        assert pool.ref.tolist() == self.ref
        words = [sum(1 << (p - w) for p in range(w, min(w + 32, len(self.ref))) if self.ref[p] == 0)
                 for w in range(0, len(self.ref), 32)]
        assert [w & 0xffffffff for w in pool.free.tolist()] == words


@pytest.mark.parametrize("pages,page,seqs,cols", [(1, 16, 1, 1), (33, 16, 5, 12), (200, 32, 40, 9), (5000, 16, 700, 30),
                                                  (70000, 16, 4096, 20)])
def test_pool_against_a_model(pages, page, seqs, cols):
    r = np.random.default_rng(pages)
    pool, model = ubw.page_pool(pages, page, seqs, cols, DEV), PoolModel(pages, page, seqs, cols)
    model.check(pool)
    steps = 60 if seqs < 1000 else 12
    for step in range(steps):
        op = r.integers(0, 4)
        if op < 2:
            room = np.where(r.random(seqs) < 0.5, r.integers(-2, 3 * page, seqs), 0).tolist()
            if step % 9 == 5:
                room[-1] = cols * page + 1
            got = ubw.pages_reserve(pool, i32(room))
            assert got.tolist() == model.reserve(room)
            take = [n + max(0, min(x, len(row) * page - n)) if r.random() < 0.8 else -1
                    for n, x, row in zip(model.len, room, model.rows)]
        elif op == 2:
            parents = np.where(r.random(seqs) < 0.3, r.integers(0, seqs + 1, seqs), -1).tolist()
            ubw.pages_fork(pool, i32(parents))
            model.fork(parents)
            model.check(pool)
            continue
        else:
            take = [int(r.integers(0, n + page)) if r.random() < 0.3 else 0 if r.random() < 0.2 else -1 for n in model.len]
        ubw.pages_trim(pool, i32(take))
        model.trim(take)
        model.check(pool)
    ubw.pages_trim(pool, i32([0] * seqs))
    model.trim([0] * seqs)
    model.check(pool)
    assert model.ref == [0] * pages


def test_pool_hands_out_everything_and_refuses_more():
    pool, model = ubw.page_pool(64, 16, 3, 64, DEV), PoolModel(64, 16, 3, 64)
    for room in ([16 * 60, 16 * 4, 0], [1, 0, 0], [16 * 60, 0, 1]):
        got = ubw.pages_reserve(pool, i32(room))
        assert got.tolist() == model.reserve(room)
        model.check(pool)
    assert pool.status.item() == ubw.PagePool.NO_PAGES
    pool.status.zero_()
    model.status = 0
    big = [2 ** 31 - 1] * 3
    ubw.pages_reserve(pool, i32(big))
    model.reserve(big)
    model.check(pool)


def test_pool_bits_past_the_last_page_are_no_pages():
    pool = ubw.page_pool(40, 16, 2, 64, DEV)
    guard = torch.full((64,), 7, dtype=torch.int32, device=DEV)
    wide = torch.cat((pool.ref, guard))   # counts behind the last page, never written
    pool = ubw.PagePool(wide[:40], pool.free, pool.table, pool.held, pool.len, pool.status, 16)
    pool.free.fill_(-1)
    ubw.pages_reserve(pool, i32([16 * 40, 0]))
    assert pool.held.tolist() == [40, 0] and pool.status.item() == 0
    ubw.pages_reserve(pool, i32([0, 1]))
    assert pool.status.item() == ubw.PagePool.NO_PAGES
    assert (wide[40:] == 7).all() and (wide[:40] == 1).all()


# ---------------------------------------------------------------------------------------------
# together

def test_a_decoding_loop():
    """Products, norm and rotation into the cache, attention of drafted trees, the o product, then the
    accepted tokens drawn together, room for the next step, and a fork that goes its own way: each
    attention against 64 bits over the tokens that were accepted, in order."""
    heads, kv, dim, page, width = 8, 2, 64, 16, 512
    rng = np.random.default_rng(21)
    parts = [make_gemv(rng, nm, n, width, 2, alpha=(0.05, 0.1)) for nm, n in (("q", heads * dim), ("k", kv * dim), ("v", kv * dim))]
    og = make_gemv(rng, "o", width, heads * dim, 2)

    def dev(a):
        a = np.ascontiguousarray(a)
        return torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a).to(DEV)

    weights = [dict(packed=ubw.pack_bases(dev(x.bits), x.nb, x.n, x.k), alpha_r=dev(x.alpha_r), alpha_c=dev(x.alpha_c), n=x.n)
               for x in parts]
    seqs, cols, pages = 4, 12, 40
    pool = ubw.page_pool(pages, page, seqs, cols, DEV)
    kc, vc = (torch.full((1, pages, kv, page, dim), math.nan, dtype=F16, device=DEV) for _ in "kv")
    cache = ubw.KVCache(kc, vc)
    freq = (10000.0 ** (-torch.arange(0, dim, 2, device=DEV, dtype=F64) / dim)).to(F32)
    w = torch.rand(dim, device=DEV, generator=gen(22)) + 0.5
    ws = ubw.tree_attn_workspace(seqs, 16, heads, kv, dim, DEV)
    told = [[] for _ in range(seqs)]   # (key, value) of each accepted token, [kv, dim] in 64 bits
    live = [True, True, True, False]
    for step in range(6):
        drafts = [int(rng.integers(0, 6)) if on else 0 for on in live]
        if step == 0:
            drafts = [5, 4, 3, 0]
        t = sum(drafts)
        if t == 0:
            continue
        room = i32(drafts)
        ubw.cache_copy_pages(cache, ubw.pages_reserve(pool, room))
        assert pool.status.item() == 0
        lens = pool.len.tolist()
        table = pool.table.cpu()
        start = [0] + list(np.cumsum(drafts))
        slots, pos, masks, trees = [], [], [], []
        for b, n in enumerate(drafts):
            tree = []
            for i in range(n):
                up = tree[int(rng.integers(0, i))] if i else []
                tree.append(up + [i])
                pos.append(lens[b] + len(up))
                slots.append(int(table[b, (lens[b] + i) // page]) * page + (lens[b] + i) % page)
                masks.append(sum(1 << j for j in tree[-1]))
            trees.append(tree)
        x = torch.from_numpy(rng.standard_normal((t, width)).astype(np.float16)).to(DEV)
        ys = [torch.empty((t, x2.n), device=DEV) for x2 in parts]
        ubw.lut_gemv_multi([d | dict(y=y) for d, y in zip(weights, ys)], x, width)
        q, k, v = (y.view(t, -1, dim) for y in ys)
        qo = ubw.qk_norm_rope(q, k, v, cache, i32(pos), i32(slots), freq, q_weight=w, k_weight=w)
        out = ubw.tree_attn(qo, cache, pool.table, i32(start), pool.len, torch.tensor(masks, device=DEV), max_tree=16,
                            workspace=ws)
        y = ubw.lut_gemv(ubw.pack_bases(dev(og.bits), og.nb, og.n, og.k), dev(og.alpha_r), dev(og.alpha_c),
                         out.view(t, -1), og.n, og.k)
        want_y = oracle.gemv(og.bits, og.alpha_r, og.alpha_c, out.view(t, -1).cpu().numpy())
        err = np.abs(y.cpu().numpy() - want_y)
        assert (err <= 1e-3 * np.maximum(np.abs(want_y), 1e-3 * np.abs(want_y).max(-1, keepdims=True))).all()
        # what is stored, then attention over accepted tokens and the drafted ones a token sees
        near(qo, *rope_reference(q, w, 1e-6, i32(pos), freq, dim, False), F16)
        flat = [c[0].transpose(1, 2).reshape(-1, kv, dim).double().cpu() for c in (kc, vc)]
        near(flat[0][slots], *rope_reference(k, w, 1e-6, i32(pos), freq, dim, False), F16)
        near(flat[1][slots], v.double().cpu(), 0 * v.double().cpu(), F16)
        accept, keep = [], []
        for b, n in enumerate(drafts):
            for i in range(n):
                r = start[b] + i
                see = told[b] + [(flat[0][slots[start[b] + j]], flat[1][slots[start[b] + j]]) for j in trees[b][i]]
                kk, vv = (torch.stack([e[z] for e in see], 1) for z in (0, 1))   # [kv, positions, dim]
                s = torch.matmul(qo[r].double().cpu().view(kv, -1, dim), kk.transpose(1, 2)) / 8
                p = torch.softmax(s, -1)
                o, size = torch.matmul(p, vv).view(heads, dim), torch.matmul(p, vv.abs()).view(heads, dim)
                reach = torch.matmul(qo[r].double().cpu().view(kv, -1, dim).abs(), kk.abs().transpose(1, 2)).amax(-1).view(heads) / 8
                lse = torch.logsumexp(s, -1).view(heads)
                check_attention(out[r:r + 1], lse[None].float(), (o[None], lse[None], size[None], reach[None]), F16, cols * page)
            path = trees[b][int(rng.integers(0, n))] if n else []
            accept.append(len(path))
            keep.append(path + [-1] * (6 - len(path)))
            told[b] += [(flat[0][slots[start[b] + j]], flat[1][slots[start[b] + j]]) for j in path]
        ubw.cache_compact(cache, pool.table, pool.len, i32(keep))
        ubw.pages_trim(pool, i32([lens[b] + a if drafts[b] else -1 for b, a in enumerate(accept)]))
        if step == 2:
            ubw.pages_fork(pool, i32([-1, -1, -1, 0]))
            told[3], live[3] = list(told[0]), True
        if step == 4:
            ubw.pages_trim(pool, i32([-1, 0, -1, -1]))
            told[1] = []
        assert pool.status.item() == 0 and pool.len.tolist() == [len(x) for x in told]


# ---------------------------------------------------------------------------------------------
# what the binding refuses

def test_binding_refusals():
    g = gen(30)
    cache = cache_of(4, 2, 16, 64, F16, g)
    q, k, v = randn((3, 4, 64), F16, g), randn((3, 2, 64), F16, g), randn((3, 2, 64), F16, g)
    pos = slots = i32([0, 1, 2])
    with pytest.raises(ValueError):
        ubw.KVCache(cache.k, cache.v, k_scale=torch.ones(2, device=DEV))
    with pytest.raises(ValueError):
        ubw.KVCache(cache.k, cache.v[:2])
    with pytest.raises(ValueError):
        ubw.KVCache(cache.k.cpu(), cache.v.cpu())
    with pytest.raises(TypeError):
        ubw.KVCache(cache.k.float(), cache.v.float())
    for bad in (dict(q=q.cpu()), dict(k=k.float()), dict(k=k[:2]), dict(v=randn((3, 3, 64), F16, g)),
                dict(q=q.transpose(0, 1)), dict(pos=pos.long()), dict(slots=slots[:2]), dict(pos=pos.cpu())):
        a = dict(q=q, k=k, v=v, pos=pos, slots=slots) | bad
        with pytest.raises((TypeError, ValueError)):
            ubw.qk_norm_rope(a["q"], a["k"], a["v"], cache, a["pos"], a["slots"], None)
    with pytest.raises(ubw.UbwError) as e:
        ubw.qk_norm_rope(q, k, v, cache, pos, slots, torch.ones(5, device=DEV))   # rot 10, halves
    assert e.value.status == ubw.UBW_EUNSUPPORTED
    table = i32([[0, 1]])
    for bad in (dict(start=i32([0])), dict(ctx=i32([1, 2])), dict(table=table.long()), dict(q=q.float()), dict(q=q[..., :32]),
                dict(masks=torch.zeros(3, device=DEV)), dict(masks=torch.zeros(2, dtype=torch.int64, device=DEV))):
        a = dict(q=q, start=i32([0, 3]), ctx=i32([1]), table=table, masks=None) | bad
        with pytest.raises((TypeError, ValueError)):
            ubw.tree_attn(a["q"], cache, a["table"], a["start"], a["ctx"], a["masks"], max_tree=3)
    with pytest.raises(ubw.UbwError):
        ubw.tree_attn(q, cache, table, i32([0, 3]), i32([1]), max_tree=65)
    with pytest.raises(ubw.UbwError):
        ubw.tree_attn(q, cache, table, i32([0, 3]), i32([1]), max_tree=3, workspace=torch.empty(8, device=DEV))
    with pytest.raises(ValueError):
        ubw.cache_copy_pages(cache, i32([0, 1]))
    with pytest.raises(ValueError):
        ubw.page_pool(0, 16, 1, 1, DEV)
