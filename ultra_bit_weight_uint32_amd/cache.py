"""Keys and values in a paged cache: the store with norm and rotation, attention over the cache, and
its pages. Thin marshalling over the calls of include/ubw.h, like the rest of the package.

A decoding step of a batch, for one layer:

    q, k, v = the products (lut_gemv_multi)                      [tokens, heads, head_dim]
    qk_norm_rope(q, k, v, cache, positions, slots, inv_freq)     keys and values into the cache
    tree_attn(q, cache, pool.table, q_start, pool.len, masks)    the input of the o product

and once per step, for all layers: pages_reserve before it, cache_compact (of the drafted tokens that
were accepted) and pages_trim behind it.

Sequences that pages_fork made share the beginning of their contexts; prefix_attn in place of tree_attn reads it once
for all of them. Long contexts need not be read whole: page_bounds after each step that fills pages (for all layers),
then per layer block_select, which names the blocks that matter to each token, and block_attn over these.

KVCache and PagePool hold the tensors and their descriptors, checked once; the calls check what
changes from call to call. Every call runs on its tensors' device, on that device's current stream.
"""
import ctypes

import torch

from . import UBW_BF16, UBW_E4M3, UBW_F16, UBW_F32, KVCacheDesc, PagePoolDesc, _check, lib

_TYPES = {torch.float32: UBW_F32, torch.float16: UBW_F16, torch.bfloat16: UBW_BF16, torch.float8_e4m3fn: UBW_E4M3}


_Tensor = torch.Tensor
_calls = {}   # library functions by name
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(fn, index, *args):
    """The call of a library function on a device, on that device's current stream."""
    f = _calls.get(fn)
    if f is None:
        f = _calls[fn] = getattr(lib(), fn)
    if _current_device() == index:
        st = f(*args, _current_stream(index))
    else:
        with torch.cuda.device(index):
            st = f(*args, _current_stream(index))
    if st:
        _check(fn, st)


def _elsewhere(t, name, index):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    raise ValueError(f"{name} is on {t.device}, the call's other tensors on cuda:{index}")


def _flat(t, name, dtype, index, numel=None, shape=None):
    """Pointer of a contiguous tensor of a dtype on the call's device. (All conditions at once first: a
    single-token call spends half its time in these questions.)"""
    if type(t) is _Tensor and t.get_device() == index and t.dtype is dtype and (numel is None or t.numel() == numel) and \
            t.is_contiguous() and (shape is None or t.shape == shape):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        _elsewhere(t, name, index)
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")
    return t.data_ptr()


def _rows(t, name, index, dim, heads=None, tokens=None, dtype=None):
    """(pointer, row stride, tokens, heads) of [tokens, heads, dim] whose heads are contiguous; rows may
    be apart (a part of a fused buffer)."""
    if not isinstance(t, _Tensor) or t.get_device() != index:
        _elsewhere(t, name, index)
    try:
        n, h, d = t.shape
    except ValueError:
        raise ValueError(f"{name} must be [tokens, heads, {dim}], got {list(t.shape)}") from None
    if d != dim or (heads is not None and h != heads) or (tokens is not None and n != tokens):
        raise ValueError(f"{name} must be [{'tokens' if tokens is None else tokens}, "
                         f"{'heads' if heads is None else heads}, {dim}], got {list(t.shape)}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    s0, s1, s2 = t.stride()
    if s2 != 1 or (h > 1 and s1 != dim):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return t.data_ptr(), s0 if n > 1 else h * dim, n, h


def _table(t, batch, index):
    """(pointer, row stride, columns) of an int32 [batch, columns] table; rows may be apart."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        _elsewhere(t, "table", index)
    if t.dim() != 2 or t.shape[0] != batch or t.dtype is not torch.int32 or t.shape[1] < 1 or \
            (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"table must be int32 [{batch}, columns] with contiguous columns")
    cols = t.shape[1]
    return t.data_ptr(), t.stride(0) if batch > 1 else cols, cols


class KVCache:
    """A paged cache: k and v [layers, pages, kv_heads, page_size, head_dim] (or without layers), fp16,
    bf16 or float8_e4m3fn, any strides with contiguous head_dim (token-major caches as views).
    k_scale, v_scale: fp32 [kv_heads], what 8-bit elements are multiplied by (default 1)."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if not k.is_cuda:
            raise ValueError("k must be on a GPU (no CPU path exists)")
        if k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must have the same shape, dtype and device")
        if k.dim() not in (4, 5):
            raise ValueError("k must be [layers, pages, kv_heads, page_size, head_dim] or without layers")
        if k.dtype not in (torch.float16, torch.bfloat16, torch.float8_e4m3fn):
            raise TypeError(f"k has dtype {k.dtype}, expected float16, bfloat16 or float8_e4m3fn")
        if k.stride(-1) != 1 or v.stride(-1) != 1:
            raise ValueError("head_dim must be contiguous")
        if k.dtype is not torch.float8_e4m3fn and (k_scale is not None or v_scale is not None):
            raise ValueError("scales belong to 8-bit caches")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device, self.index, self.dtype = k.device, k.get_device(), k.dtype
        k5, v5 = (x if x.dim() == 5 else x[None] for x in (k, v))
        self.layers, self.pages, self.kv_heads, self.page_size, self.head_dim = k5.shape
        d = KVCacheDesc()
        d.k, d.v, d.dtype = k.data_ptr(), v.data_ptr(), _TYPES[k.dtype]
        d.layers, d.pages, d.page_size, d.kv_heads, d.head_dim = (self.layers, self.pages, self.page_size,
                                                                  self.kv_heads, self.head_dim)
        d.k_stride[:], d.v_stride[:] = k5.stride()[:4], v5.stride()[:4]
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if s is not None:
                setattr(d, name, _flat(s, name, torch.float32, self.index, self.kv_heads))
        self.desc, self.ref = d, ctypes.byref(d)

    def layer(self, i):
        """The cache of one layer, as the calls of that layer take it."""
        if self.k.dim() != 5:
            raise ValueError("this cache has one layer")
        return KVCache(self.k[i], self.v[i], self.k_scale, self.v_scale)


def qk_norm_rope(q, k, v, cache, positions, slots, inv_freq, q_weight=None, k_weight=None, eps=1e-6,
                 interleaved=False, out=None, out_dtype=None):
    """Norms of queries and keys for each head (weights fp32 [head_dim], None: no norm), rotation at
    positions (int32 [tokens]) by inv_freq (fp32 [rot / 2], None: no rotation), keys and values stored
    at slots (int32 [tokens]; outside the cache: not stored) of the cache. q [tokens, heads, head_dim],
    k, v [tokens, kv_heads, head_dim] in fp32, fp16 or bf16. Returns the queries [tokens, heads,
    head_dim] in out (or a new tensor of out_dtype; default the cache's type, fp16 for 8 bits)."""
    dev, dim, kvh = cache.index, cache.head_dim, cache.kv_heads
    dtype = q.dtype
    qp, ldq, t, heads = _rows(q, "q", dev, dim)
    kp, ldk, _, _ = _rows(k, "k", dev, dim, kvh, t, dtype)
    vp, ldv, _, _ = _rows(v, "v", dev, dim, kvh, t, dtype)
    if dtype is torch.float8_e4m3fn or dtype not in _TYPES:
        raise TypeError(f"q has dtype {dtype}, expected float32, float16 or bfloat16")
    if out is None:
        if out_dtype is None:
            out_dtype = torch.float16 if cache.dtype is torch.float8_e4m3fn else cache.dtype
        out = torch.empty((t, heads, dim), dtype=out_dtype, device=cache.device)
    op, ldo, _, _ = _rows(out, "out", dev, dim, heads, t)
    if out.dtype is not torch.float16 and out.dtype is not torch.bfloat16:
        raise TypeError(f"out has dtype {out.dtype}, expected float16 or bfloat16")
    f32, i32 = torch.float32, torch.int32
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    _launch("ubw_qk_norm_rope", dev, cache.ref, qp, ldq, kp, ldk, vp, ldv, _TYPES[dtype], t, heads,
            None if q_weight is None else _flat(q_weight, "q_weight", f32, dev, dim),
            None if k_weight is None else _flat(k_weight, "k_weight", f32, dev, dim), eps,
            None if rot == 0 else _flat(inv_freq, "inv_freq", f32, dev), rot, 1 if interleaved else 0,
            _flat(positions, "positions", i32, dev, t), _flat(slots, "slots", i32, dev, t), op, _TYPES[out.dtype], ldo)
    return out


def tree_attn_workspace(batch, max_tree, heads, kv_heads, head_dim, device="cuda"):
    """Scratch for tree_attn calls of up to these sizes (reusable on one stream)."""
    n = ctypes.c_size_t()
    _check("ubw_tree_attn_workspace_bytes",
           lib().ubw_tree_attn_workspace_bytes(batch, max_tree, heads, kv_heads, head_dim, ctypes.byref(n)))
    return torch.empty(-(-n.value // 4), dtype=torch.float32, device=device)


def _attn_args(q, cache, table, q_start, ctx_len, masks, scale, out, lse):
    """What the attention calls check alike: (out, (q .. table_cols), masks, scale, (out, ldo, lse))."""
    dev, dim = cache.index, cache.head_dim
    qp, ldq, t, heads = _rows(q, "q", dev, dim)
    dtype = q.dtype
    if dtype is not torch.float16 and dtype is not torch.bfloat16:
        raise TypeError(f"q has dtype {dtype}, expected float16 or bfloat16")
    if out is None:
        out = torch.empty((t, heads, dim), dtype=dtype, device=cache.device)
    op, ldo, _, _ = _rows(out, "out", dev, dim, heads, t, dtype)
    i32 = torch.int32
    batch = ctx_len.numel()
    tp, ld_table, cols = _table(table, batch, dev)
    if masks is not None:
        if masks.dtype is not torch.int64 and masks.dtype is not torch.uint64:
            raise TypeError(f"masks has dtype {masks.dtype}, expected int64 or uint64")
        masks = _flat(masks, "masks", masks.dtype, dev, t)
    return (out, (cache.ref, qp, _TYPES[dtype], ldq, t, heads, _flat(q_start, "q_start", i32, dev, batch + 1),
                  _flat(ctx_len, "ctx_len", i32, dev), batch, tp, ld_table, cols),
            (masks, dim ** -0.5 if scale is None else scale, op, ldo,
             None if lse is None else _flat(lse, "lse", torch.float32, dev, shape=(t, heads))))


def _scratch(workspace, index):
    """(pointer, bytes) of a workspace, or of none."""
    return (None, 0) if workspace is None else (_flat(workspace, "workspace", workspace.dtype, index), workspace.nbytes)


def tree_attn(q, cache, table, q_start, ctx_len, masks=None, *, max_tree, max_len=0, scale=None, out=None, lse=None,
              workspace=None):
    """Attention of each sequence's new tokens (one, or a tree of up to 64 drafted ones) over its context
    in the cache and over one another. q [tokens, heads, head_dim]; table int32 [batch, columns] (rows
    may be apart); q_start int32 [batch + 1]; ctx_len int32 [batch]; masks int64 or uint64 [tokens], bit
    j of a token's: it sees token j of its tree (None: those up to itself). max_tree: the most tokens a
    sequence has; max_len: the longest context plus tokens (0: unknown). lse: None or fp32 [tokens,
    heads] to be written. workspace: tree_attn_workspace() (None: long contexts are not split over
    workgroups). Returns out [tokens, heads, head_dim] in q's type."""
    out, first, last = _attn_args(q, cache, table, q_start, ctx_len, masks, scale, out, lse)
    _launch("ubw_tree_attn", cache.index, *first, max_tree, max_len, *last, *_scratch(workspace, cache.index))
    return out


def prefix_attn_workspace(batch, groups, tokens, max_tree, heads, kv_heads, head_dim, device="cuda"):
    """Scratch for prefix_attn calls of these sizes, with this many tokens in all or fewer (reusable on one stream)."""
    n = ctypes.c_size_t()
    _check("ubw_prefix_attn_workspace_bytes", lib().ubw_prefix_attn_workspace_bytes(
        batch, groups, tokens, max_tree, heads, kv_heads, head_dim, ctypes.byref(n)))
    return torch.empty(-(-n.value // 4), dtype=torch.float32, device=device)


def prefix_attn(q, cache, table, q_start, ctx_len, group_start, prefix_len, masks=None, *, max_tree, workspace, max_len=0,
                scale=None, out=None, lse=None):
    """tree_attn for sequences that have the beginning of their contexts in common: the sequences group_start[g] ..
    group_start[g + 1] - 1 (int32 [groups + 1], ascending) hold the same keys and values at the first prefix_len[g]
    (int32 [groups]) positions, which are read once for all of them, by the table row of the first sequence that has
    tokens. Sequences in no group have their contexts for themselves, and so has a batch of short ones, where that takes
    less time (max_len, or else the table's width, tells). workspace: prefix_attn_workspace(); the other arguments as
    tree_attn's."""
    out, first, last = _attn_args(q, cache, table, q_start, ctx_len, masks, scale, out, lse)
    i32, dev = torch.int32, cache.index
    groups = prefix_len.numel()
    _launch("ubw_prefix_attn", dev, *first, _flat(group_start, "group_start", i32, dev, groups + 1),
            _flat(prefix_len, "prefix_len", i32, dev), groups, max_tree, max_len, *last, *_scratch(workspace, dev))
    return out


def page_bounds(cache, bounds, table, start, stop, *, max_new=0):
    """The smallest and the largest key element of every dim, for the pages that were filled when the sequences grew
    from start to stop positions (int32 [batch] each): the columns start // page_size .. stop // page_size - 1 of
    table, in every layer. bounds [layers, pages, kv_heads, 2, head_dim] (without layers where the cache has none), of
    the cache's type, takes them at [..., 0, :] and [..., 1, :]; other pages' stay. max_new: the most positions a
    sequence grew by (0: unknown)."""
    dev, i32 = cache.index, torch.int32
    shape = cache.k.shape[:-2] + (2, cache.head_dim)
    batch = start.numel()
    tp, ld_table, cols = _table(table, batch, dev)
    _launch("ubw_page_bounds", dev, cache.ref, _flat(bounds, "bounds", cache.dtype, dev, shape=shape), tp, ld_table, cols,
            _flat(start, "start", i32, dev), _flat(stop, "stop", i32, dev, batch), batch, max_new)


def block_select_workspace(tokens, kv_heads, max_blocks, device="cuda"):
    """Scratch for block_select calls of up to this many tokens over tables of up to max_blocks columns (reusable on one
    stream)."""
    n = ctypes.c_size_t()
    _check("ubw_block_select_workspace_bytes",
           lib().ubw_block_select_workspace_bytes(tokens, kv_heads, max_blocks, ctypes.byref(n)))
    return torch.empty(-(-n.value // 8), dtype=torch.int64, device=device)


def block_select(q, bounds, table, q_start, ctx_len, count, *, page_size, max_tree, workspace, first=1, last=1, max_len=0,
                 out=None):
    """For each token and key/value head the `count` whole blocks (pages) of its sequence's context that its query heads
    may score highest, by the keys' bounds [pages, kv_heads, 2, head_dim] of one layer (page_bounds()); the `first`
    and the `last` whole blocks are always among them. Returns out, int32 [tokens, kv_heads, count]: block indices
    (columns of table), ascending, -1 behind them where the context has fewer. workspace: block_select_workspace();
    the other arguments as tree_attn's."""
    if not isinstance(bounds, _Tensor) or bounds.dim() != 4 or bounds.shape[2] != 2 or not bounds.is_cuda:
        raise ValueError("bounds must be a GPU tensor [pages, kv_heads, 2, head_dim]")
    dev, i32 = bounds.get_device(), torch.int32
    pages, kv, _, dim = bounds.shape
    dtype = bounds.dtype
    if dtype not in _TYPES or dtype is torch.float32:
        raise TypeError(f"bounds has dtype {dtype}, expected float16, bfloat16 or float8_e4m3fn")
    qp, ldq, t, heads = _rows(q, "q", dev, dim)
    if q.dtype is not torch.float16 and q.dtype is not torch.bfloat16:
        raise TypeError(f"q has dtype {q.dtype}, expected float16 or bfloat16")
    batch = ctx_len.numel()
    tp, ld_table, cols = _table(table, batch, dev)
    if out is None:
        out = torch.empty((t, kv, max(count, 0)), dtype=i32, device=bounds.device)
    _launch("ubw_block_select", dev, _flat(bounds, "bounds", dtype, dev), _TYPES[dtype], pages, page_size, kv, dim, qp,
            _TYPES[q.dtype], ldq, t, heads, _flat(q_start, "q_start", i32, dev, batch + 1), _flat(ctx_len, "ctx_len", i32, dev),
            batch, tp, ld_table, cols, max_tree, max_len, count, first, last,
            _flat(out, "out", i32, dev, shape=(t, kv, count)), *_scratch(workspace, dev))
    return out


def block_attn_workspace(tokens, heads, kv_heads, head_dim, device="cuda"):
    """Scratch for block_attn calls of up to this many tokens (reusable on one stream)."""
    n = ctypes.c_size_t()
    _check("ubw_block_attn_workspace_bytes",
           lib().ubw_block_attn_workspace_bytes(tokens, heads, kv_heads, head_dim, ctypes.byref(n)))
    return torch.empty(-(-n.value // 4), dtype=torch.float32, device=device)


def block_attn(q, cache, table, q_start, ctx_len, blocks, masks=None, *, max_tree, scale=None, out=None, lse=None,
               workspace=None):
    """tree_attn where a token sees, of its sequence's whole blocks (pages), only those in its list: blocks int32
    [tokens, kv_heads, count], ascending block indices, as block_select() gives them; a list ends at its first entry that
    does not ascend or is no whole block of the context. The page on which the context ends and the tokens behind it
    are seen as in tree_attn. workspace: block_attn_workspace() (None: lists are not split over workgroups)."""
    out, head, rest = _attn_args(q, cache, table, q_start, ctx_len, masks, scale, out, lse)
    dev = cache.index
    bp = _flat(blocks, "blocks", torch.int32, dev)
    if blocks.dim() != 3 or blocks.shape[0] != q.shape[0] or blocks.shape[1] != cache.kv_heads:
        raise ValueError(f"blocks must be [{q.shape[0]}, {cache.kv_heads}, count], got {list(blocks.shape)}")
    _launch("ubw_block_attn", dev, *head, bp, blocks.shape[2], max_tree, *rest, *_scratch(workspace, dev))
    return out


def cache_copy_pages(cache, pairs):
    """Page pairs[i, 0] copied to page pairs[i, 1] (int32 [count, 2]), keys and values of every layer.
    Pairs with an entry outside the cache's pages, as (-1, -1), are skipped."""
    p = _flat(pairs, "pairs", torch.int32, cache.index)
    if pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError(f"pairs must be [count, 2], got {list(pairs.shape)}")
    _launch("ubw_cache_copy_pages", cache.index, cache.ref, p, pairs.shape[0])


def cache_compact(cache, table, ctx_len, keep):
    """Keys and values at position ctx_len[b] + keep[b, i] moved to ctx_len[b] + i in every layer, for
    i = 0, 1, ... up to the first entry of keep (int32 [batch, width]) that does not ascend from 0."""
    dev, i32 = cache.index, torch.int32
    kp = _flat(keep, "keep", i32, dev)
    if keep.dim() != 2:
        raise ValueError(f"keep must be [batch, width], got {list(keep.shape)}")
    batch, width = keep.shape
    tp, ld_table, cols = _table(table, batch, dev)
    _launch("ubw_cache_compact", dev, cache.ref, tp, ld_table, cols, _flat(ctx_len, "ctx_len", i32, dev, batch), kp,
            width, batch)


class PagePool:
    """Pages shared out over sequences, in device memory (ubw_page_pool of include/ubw.h): ref int32
    [pages], free int32 [ceil(pages / 32)] (a bit set), table int32 [seqs, max_pages], held and len
    int32 [seqs], status int32 [1]. page_pool() makes an empty one."""

    NO_PAGES, NOT_SERVED = 1, 2   # bits of status

    def __init__(self, ref, free, table, held, len, status, page_size):
        if not ref.is_cuda:
            raise ValueError("ref must be on a GPU (no CPU path exists)")
        self.ref, self.free, self.table, self.held, self.len, self.status = ref, free, table, held, len, status
        self.device, self.index, self.page_size = ref.device, ref.get_device(), page_size
        self.pages, (self.seqs, self.max_pages) = ref.numel(), table.shape
        i32, dev = torch.int32, self.index
        d = PagePoolDesc()
        d.ref = _flat(ref, "ref", i32, dev)
        d.free_bits = _flat(free, "free", i32, dev, numel=-(-self.pages // 32))
        d.table = _flat(table, "table", i32, dev)
        d.held = _flat(held, "held", i32, dev, numel=self.seqs)
        d.len = _flat(len, "len", i32, dev, numel=self.seqs)
        d.status = _flat(status, "status", i32, dev, numel=1)
        d.pages, d.page_size, d.seqs, d.max_pages = self.pages, page_size, self.seqs, self.max_pages
        self.desc, self.byref = d, ctypes.byref(d)


def page_pool(pages, page_size, seqs, max_pages, device="cuda"):
    """An empty pool: every page free, no sequence holding any."""
    if pages < 1 or seqs < 1 or max_pages < 1:
        raise ValueError("pages, seqs and max_pages must be positive")
    new = [torch.empty(n, dtype=torch.int32, device=device)
           for n in (pages, -(-pages // 32), (seqs, max_pages), seqs, seqs, 1)]
    pool = PagePool(*new, page_size)
    _launch("ubw_pages_init", pool.index, pool.byref)
    return pool


def pages_trim(pool, new_len):
    """len[s] = new_len[s] where that is not negative (int32 [seqs]), the pages behind it given back."""
    _launch("ubw_pages_trim", pool.index, pool.byref, _flat(new_len, "new_len", torch.int32, pool.index, pool.seqs))


def pages_fork(pool, parents):
    """Sequence s becomes a copy of parents[s] where that is not negative (int32 [seqs]), by sharing."""
    _launch("ubw_pages_fork", pool.index, pool.byref, _flat(parents, "parents", torch.int32, pool.index, pool.seqs))


def pages_reserve(pool, room, pairs=None):
    """Pages for room[s] more tokens of each sequence (int32 [seqs]). Returns pairs, int32 [seqs, 2]:
    (old, new) where a sequence got its own copy of a shared page, to be passed to cache_copy_pages
    before the pool's next call; (-1, -1) elsewhere."""
    p = _flat(room, "room", torch.int32, pool.index, pool.seqs)
    if pairs is None:
        pairs = torch.empty((pool.seqs, 2), dtype=torch.int32, device=pool.device)
    _launch("ubw_pages_reserve", pool.index, pool.byref, p,
            _flat(pairs, "pairs", torch.int32, pool.index, shape=(pool.seqs, 2)))
    return pairs
