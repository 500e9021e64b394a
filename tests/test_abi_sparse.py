"""CPU-only checks of attention over shared prefixes and over selected blocks: every refusal happens on the host
before anything is enqueued, and calls with nothing to do return without touching the device (no GPU needed)."""
import ctypes

import pytest

import ultra_bit_weight_uint32_amd as ubw
from test_abi_cache import (BAD_CACHES, BF16, E4M3, EALIGN, EINVAL, ERANGE, ESIZE, EUNSUP, F16, F32, FAKE, OK, cache,
                            split)

BIG = 1 << 40   # bytes that no workspace needs more than


def prefix(**kw):
    c, kw = split(kw)
    a = dict(cache=cache(**c), q=FAKE, q_dtype=F16, ldq=2048, tokens=3, heads=16, start=FAKE, ctx=FAKE, batch=2,
             table=FAKE, ld_table=10, cols=10, group_start=FAKE, prefix_len=FAKE, groups=1, max_tree=2, max_len=0, masks=None,
             scale=0.1, out=FAKE, ldo=2048, lse=None, ws=FAKE, wsb=64, stream=None)
    a.update(kw)
    return ubw.lib().ubw_prefix_attn(*a.values())


def bounds(**kw):
    c, kw = split(kw)
    a = dict(cache=cache(**c), bounds=FAKE, table=FAKE, ld_table=10, cols=10, start=FAKE, stop=FAKE, batch=2, max_new=0,
             stream=None)
    a.update(kw)
    return ubw.lib().ubw_page_bounds(*a.values())


def select(**kw):
    a = dict(bounds=FAKE, dtype=F16, pages=10, page_size=16, kv_heads=8, head_dim=128, q=FAKE, q_dtype=F16, ldq=2048,
             tokens=3, heads=16, start=FAKE, ctx=FAKE, batch=2, table=FAKE, ld_table=10, cols=10, max_tree=2, max_len=0,
             count=4, first=1, last=1, blocks=FAKE, ws=FAKE, wsb=64, stream=None)
    a.update(kw)
    return ubw.lib().ubw_block_select(*a.values())


def attn(**kw):
    c, kw = split(kw)
    a = dict(cache=cache(**c), q=FAKE, q_dtype=F16, ldq=2048, tokens=3, heads=16, start=FAKE, ctx=FAKE, batch=2,
             table=FAKE, ld_table=10, cols=10, blocks=FAKE, count=4, max_tree=2, masks=None, scale=0.1, out=FAKE, ldo=2048,
             lse=None, ws=FAKE, wsb=64, stream=None)
    a.update(kw)
    return ubw.lib().ubw_block_attn(*a.values())


@pytest.mark.parametrize("call", [prefix, bounds, attn])
@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(call, kw, status):
    assert call(**kw) == status


# what both attention calls refuse, as tree attention does (the workspace of 64 bytes is too small for all)
@pytest.mark.parametrize("call", [prefix, attn])
@pytest.mark.parametrize("kw,status", [
    (dict(), ESIZE), (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(start=None), EINVAL), (dict(ctx=None), EINVAL),
    (dict(table=None), EINVAL), (dict(cols=0), EINVAL), (dict(ld_table=9), EINVAL), (dict(tokens=-1), EINVAL),
    (dict(batch=-1), EINVAL), (dict(heads=0), EINVAL), (dict(heads=12), EINVAL), (dict(max_tree=0), EINVAL),
    (dict(scale=0.0), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL),
    (dict(q_dtype=F32), EUNSUP), (dict(q_dtype=E4M3), EUNSUP), (dict(q_dtype=BF16), EUNSUP), (dict(c_dtype=BF16), EUNSUP),
    (dict(batch=4097), ERANGE), (dict(max_tree=65), ERANGE), (dict(tokens=(1 << 24) + 1), ERANGE), (dict(q=FAKE + 8), EALIGN),
    (dict(ldq=2052), EALIGN), (dict(ldo=2049), EALIGN), (dict(ldq=1024), EINVAL), (dict(masks=FAKE + 4), EALIGN),
    (dict(lse=FAKE + 2), EALIGN), (dict(start=FAKE + 2), EALIGN), (dict(ctx=FAKE + 1), EALIGN), (dict(table=FAKE + 2), EALIGN),
    (dict(ws=FAKE + 4), EALIGN), (dict(ws=None), EINVAL), (dict(cols=1 << 25, ld_table=1 << 25), ERANGE),
    (dict(c_page_size=1024, cols=1 << 21, ld_table=1 << 21), ERANGE), (dict(tokens=0, q=None, out=None, start=None), OK),
    (dict(batch=0, start=None, ctx=None, table=None), OK),
])
def test_attention_refuses(call, kw, status):
    assert call(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(group_start=None), EINVAL), (dict(prefix_len=None), EINVAL), (dict(groups=-1), EINVAL), (dict(max_len=-1), EINVAL),
    (dict(groups=4097), ERANGE), (dict(group_start=FAKE + 2), EALIGN), (dict(prefix_len=FAKE + 1), EALIGN),
    (dict(groups=0, group_start=None, prefix_len=None), ESIZE), (dict(ws=None, wsb=0), EINVAL),
    (dict(tokens=1 << 24, heads=1024, c_kv_heads=1, ldq=131072, ldo=131072), ERANGE),
])
def test_prefix_refuses(kw, status):
    assert prefix(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(bounds=None), EINVAL), (dict(table=None), EINVAL), (dict(start=None), EINVAL), (dict(stop=None), EINVAL),
    (dict(cols=0), EINVAL), (dict(ld_table=9), EINVAL), (dict(batch=-1), EINVAL), (dict(max_new=-1), EINVAL),
    (dict(batch=4097), ERANGE), (dict(bounds=FAKE + 8), EALIGN), (dict(start=FAKE + 2), EALIGN), (dict(stop=FAKE + 3), EALIGN),
    (dict(table=FAKE + 1), EALIGN), (dict(cols=1 << 25, ld_table=1 << 25), ERANGE), (dict(batch=0, table=None, bounds=None), OK),
])
def test_bounds_refuse(kw, status):
    assert bounds(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(), ESIZE), (dict(bounds=None), EINVAL), (dict(q=None), EINVAL), (dict(start=None), EINVAL), (dict(ctx=None), EINVAL),
    (dict(table=None), EINVAL), (dict(blocks=None), EINVAL), (dict(ws=None), EINVAL), (dict(ws=None, wsb=0), EINVAL),
    (dict(pages=0), EINVAL), (dict(kv_heads=0), EINVAL), (dict(heads=0), EINVAL), (dict(heads=12), EINVAL),
    (dict(tokens=-1), EINVAL), (dict(batch=-1), EINVAL), (dict(max_tree=0), EINVAL), (dict(max_len=-1), EINVAL),
    (dict(count=0), EINVAL), (dict(first=-1), EINVAL), (dict(last=-1), EINVAL), (dict(first=3, last=2), EINVAL),
    (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), EINVAL), (dict(first=2, last=2), ESIZE),
    (dict(cols=0), EINVAL), (dict(ld_table=9), EINVAL), (dict(ldq=1024), EINVAL),
    (dict(dtype=F32), EUNSUP), (dict(q_dtype=F32), EUNSUP), (dict(q_dtype=E4M3), EUNSUP), (dict(q_dtype=BF16), EUNSUP),
    (dict(dtype=BF16), EUNSUP), (dict(dtype=E4M3, q_dtype=BF16), ESIZE), (dict(head_dim=96), EUNSUP),
    (dict(page_size=8), EUNSUP), (dict(page_size=24), EUNSUP), (dict(page_size=2048), EUNSUP),
    (dict(pages=(1 << 24) + 1), ERANGE), (dict(pages=1 << 22, page_size=1024), ERANGE), (dict(batch=4097), ERANGE),
    (dict(max_tree=65), ERANGE), (dict(tokens=(1 << 24) + 1), ERANGE), (dict(count=(1 << 20) + 1), ERANGE),
    (dict(heads=2048, kv_heads=1, ldq=1 << 20), ERANGE), (dict(cols=1 << 25, ld_table=1 << 25), ERANGE),
    (dict(bounds=FAKE + 8), EALIGN), (dict(q=FAKE + 2), EALIGN), (dict(ldq=2052), EALIGN), (dict(start=FAKE + 2), EALIGN),
    (dict(ctx=FAKE + 1), EALIGN), (dict(blocks=FAKE + 2), EALIGN), (dict(table=FAKE + 2), EALIGN), (dict(ws=FAKE + 8), EALIGN),
    (dict(tokens=0, q=None, blocks=None, ws=None), OK), (dict(batch=0, table=None), OK),
])
def test_select_refuses(kw, status):
    assert select(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(blocks=None), EINVAL), (dict(count=-1), EINVAL), (dict(blocks=FAKE + 2), EALIGN), (dict(count=(1 << 20) + 1), ERANGE),
    (dict(count=1 << 20, c_page_size=1024), ERANGE), (dict(count=0, blocks=None), ESIZE), (dict(ws=None, wsb=4), EINVAL),
])
def test_block_attention_refuses(kw, status):
    assert attn(**kw) == status


def test_workspace_sizes():
    L, n = ubw.lib(), ctypes.c_size_t()

    def prefix_bytes(batch, groups, tokens, tree, heads=64, kv=8, dim=128):
        st = L.ubw_prefix_attn_workspace_bytes(batch, groups, tokens, tree, heads, kv, dim, ctypes.byref(n))
        return n.value if st == OK else st

    def block_bytes(tokens, heads=64, kv=8, dim=128):
        st = L.ubw_block_attn_workspace_bytes(tokens, heads, kv, dim, ctypes.byref(n))
        return n.value if st == OK else st

    def select_bytes(tokens, kv=8, blocks=100):
        st = L.ubw_block_select_workspace_bytes(tokens, kv, blocks, ctypes.byref(n))
        return n.value if st == OK else st

    # what serves a call serves every smaller one
    base = dict(batch=8, groups=2, tokens=64, tree=8)
    for more in (dict(batch=9), dict(groups=3), dict(tokens=65), dict(tree=9), dict(batch=4096, groups=4096, tokens=4096, tree=64)):
        assert 0 < prefix_bytes(**base) <= prefix_bytes(**(base | more)) < BIG, more
    assert prefix_bytes(0, 0, 0, 1) > 0
    sizes = [block_bytes(t) for t in (0, 1, 2, 7, 64, 1000)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert select_bytes(3, 8, 100) == 3 * 8 * 100 * 8 and select_bytes(0) == 0
    for bad, st in ((dict(batch=-1), EINVAL), (dict(groups=-1), EINVAL), (dict(tokens=-1), EINVAL), (dict(tree=0), EINVAL),
                    (dict(heads=63), EINVAL), (dict(dim=80), EUNSUP), (dict(tree=65), ERANGE), (dict(batch=4097), ERANGE),
                    (dict(groups=4097), ERANGE), (dict(tokens=1 << 24, heads=1024, kv=1), ERANGE)):
        assert prefix_bytes(**(base | bad)) == st, bad
    for bad, st in ((dict(tokens=-1), EINVAL), (dict(tokens=1, heads=9), EINVAL), (dict(tokens=1, dim=32), EUNSUP),
                    (dict(tokens=(1 << 24) + 1), ERANGE), (dict(tokens=1, heads=2048, kv=1), ERANGE)):
        assert block_bytes(**bad) == st, bad
    for bad, st in ((dict(tokens=-1), EINVAL), (dict(tokens=1, kv=0), EINVAL), (dict(tokens=1, blocks=0), EINVAL),
                    (dict(tokens=1, kv=5000), ERANGE), (dict(tokens=1, blocks=1 << 25), ERANGE)):
        assert select_bytes(**bad) == st, bad
    assert L.ubw_prefix_attn_workspace_bytes(1, 1, 1, 1, 1, 1, 64, None) == EINVAL
    assert L.ubw_block_attn_workspace_bytes(1, 1, 1, 64, None) == EINVAL
    assert L.ubw_block_select_workspace_bytes(1, 1, 1, None) == EINVAL
