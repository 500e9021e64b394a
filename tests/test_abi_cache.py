"""CPU-only checks of the key/value cache calls: every refusal happens on the host before anything is
enqueued, and calls with nothing to do return without touching the device (no GPU needed)."""
import ctypes

import pytest

import ultra_bit_weight_uint32_amd as ubw

OK, EINVAL, EUNSUP, EALIGN, ERANGE, ESIZE = 0, -1, -2, -3, -4, -6
FAKE, OTHER = 0x10000, 0x20000          # 16-byte aligned, never dereferenced on these paths
F32, F16, BF16, E4M3 = 0, 1, 2, 3
CACHE_FIELDS = ("dtype", "layers", "pages", "page_size", "kv_heads", "head_dim")


def cache(**kw):
    d = ubw.KVCacheDesc()
    d.k, d.v = kw.pop("k", FAKE), kw.pop("v", OTHER)
    for f, x in zip(CACHE_FIELDS, (F16, 2, 10, 16, 8, 128)):
        setattr(d, f, kw.pop(f, x))
    row = max(d.head_dim, 1)
    st = [d.pages * d.kv_heads * d.page_size * row, d.kv_heads * d.page_size * row, d.page_size * row, row]
    for i, x in kw.pop("strides", {}).items():
        st[i] = x
    d.k_stride[:], d.v_stride[:] = st, st
    assert not kw
    return ctypes.byref(d)


def split(kw):
    names = CACHE_FIELDS + ("k", "v", "strides")
    return {k[2:]: v for k, v in kw.items() if k[:2] == "c_" and k[2:] in names}, \
        {k: v for k, v in kw.items() if k[:2] != "c_"}


def rope(**kw):
    c, kw = split(kw)
    a = dict(cache=cache(**c), q=FAKE, ldq=1024, k=FAKE, ldk=1024, v=FAKE, ldv=1024, in_dtype=F32, tokens=3, heads=8,
             qw=None, kw=None, eps=1e-6, freq=FAKE, rot=128, inter=0, pos=FAKE, slots=FAKE, out=FAKE, out_dtype=F16,
             ldo=1024, stream=None)
    a.update(kw)
    return ubw.lib().ubw_qk_norm_rope(*a.values())


def attn(**kw):
    c, kw = split(kw)
    a = dict(cache=cache(**c), q=FAKE, q_dtype=F16, ldq=2048, tokens=3, heads=16, start=FAKE, ctx=FAKE, batch=2,
             table=FAKE, ld_table=10, cols=10, max_tree=2, max_len=0, masks=None, scale=0.1, out=FAKE, ldo=2048, lse=None,
             ws=None, wsb=0, stream=None)
    a.update(kw)
    return ubw.lib().ubw_tree_attn(*a.values())


def copy(**kw):
    c, kw = split(kw)
    a = dict(cache=cache(**c), pairs=FAKE, count=2, stream=None)
    a.update(kw)
    return ubw.lib().ubw_cache_copy_pages(*a.values())


def compact(**kw):
    c, kw = split(kw)
    a = dict(cache=cache(**c), table=FAKE, ld=10, cols=10, ctx=FAKE, keep=FAKE, width=4, batch=2, stream=None)
    a.update(kw)
    return ubw.lib().ubw_cache_compact(*a.values())


# what every call refuses of a cache
BAD_CACHES = [
    (dict(cache=None), EINVAL), (dict(c_k=None), EINVAL), (dict(c_v=None), EINVAL), (dict(c_layers=0), EINVAL),
    (dict(c_pages=0), EINVAL), (dict(c_kv_heads=0), EINVAL), (dict(c_dtype=F32), EUNSUP), (dict(c_dtype=9), EUNSUP),
    (dict(c_head_dim=96), EUNSUP), (dict(c_head_dim=512), EUNSUP), (dict(c_page_size=8), EUNSUP),
    (dict(c_page_size=48), EUNSUP), (dict(c_page_size=2048), EUNSUP), (dict(c_k=FAKE + 8), EALIGN),
    (dict(c_v=FAKE + 2), EALIGN), (dict(c_strides={3: 132}), EALIGN), (dict(c_strides={2: -128}), ERANGE),
    (dict(c_strides={3: 64}), EINVAL), (dict(c_strides={3: 1 << 26}), ERANGE), (dict(c_strides={1: 1 << 50}), ERANGE),
    (dict(c_pages=1 << 25), ERANGE), (dict(c_pages=1 << 22, c_page_size=1024), ERANGE),
]


@pytest.mark.parametrize("call", [rope, attn, copy, compact])
@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(call, kw, status):
    assert call(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), EINVAL), (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(out=None), EINVAL),
    (dict(pos=None), EINVAL), (dict(slots=None), EINVAL), (dict(freq=None), EINVAL), (dict(tokens=-1), EINVAL),
    (dict(heads=0), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL),
    (dict(in_dtype=E4M3), EUNSUP), (dict(in_dtype=7), EUNSUP), (dict(out_dtype=F32), EUNSUP), (dict(out_dtype=E4M3), EUNSUP),
    (dict(rot=130), EUNSUP), (dict(rot=63, inter=1), EUNSUP), (dict(rot=24), EUNSUP), (dict(rot=-2), EINVAL),
    (dict(q=FAKE + 4), EALIGN), (dict(ldk=1025), EALIGN), (dict(in_dtype=F16, ldv=1028), EALIGN), (dict(ldo=1028), EALIGN),
    (dict(qw=FAKE + 4), EALIGN), (dict(kw=FAKE + 8), EALIGN), (dict(ldq=512), EINVAL), (dict(ldo=1016), EINVAL),
    (dict(tokens=1 << 24), ERANGE), (dict(tokens=0, pos=None, slots=None, q=None, out=None), OK),
])
def test_rope_refuses(kw, status):
    assert rope(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(start=None), EINVAL), (dict(ctx=None), EINVAL),
    (dict(table=None), EINVAL), (dict(cols=0), EINVAL), (dict(ld_table=9), EINVAL), (dict(tokens=-1), EINVAL),
    (dict(batch=-1), EINVAL), (dict(heads=0), EINVAL), (dict(heads=12), EINVAL), (dict(max_tree=0), EINVAL),
    (dict(max_len=-1), EINVAL), (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(scale=float("inf")), EINVAL), (dict(q_dtype=F32), EUNSUP), (dict(q_dtype=E4M3), EUNSUP),
    (dict(q_dtype=BF16), EUNSUP), (dict(c_dtype=BF16), EUNSUP), (dict(batch=4097), ERANGE), (dict(max_tree=65), ERANGE),
    (dict(tokens=(1 << 24) + 1), ERANGE), (dict(q=FAKE + 8), EALIGN), (dict(ldq=2052), EALIGN), (dict(ldo=2049), EALIGN),
    (dict(ldq=1024), EINVAL), (dict(masks=FAKE + 4), EALIGN), (dict(lse=FAKE + 2), EALIGN), (dict(ws=None, wsb=4), EINVAL),
    (dict(ws=FAKE + 4, wsb=1 << 30), EALIGN), (dict(ws=FAKE, wsb=64), ESIZE), (dict(cols=1 << 25, ld_table=1 << 25), ERANGE),
    (dict(c_page_size=1024, cols=1 << 21, ld_table=1 << 21), ERANGE),
    (dict(tokens=0, q=None, out=None, start=None), OK), (dict(batch=0, start=None, ctx=None, table=None), OK),
])
def test_attention_refuses(kw, status):
    assert attn(**kw) == status


def test_attention_workspace_size():
    n, L = ctypes.c_size_t(), ubw.lib()
    fn = L.ubw_tree_attn_workspace_bytes
    sizes = []
    for tree in (1, 2, 4, 8, 16, 32, 64):
        assert fn(4, tree, 64, 8, 128, ctypes.byref(n)) == OK and n.value > 0
        sizes.append(n.value)
    assert sizes == sorted(sizes)
    assert fn(0, 1, 8, 8, 64, ctypes.byref(n)) == OK
    assert fn(4, 1, 64, 8, 128, None) == EINVAL
    assert fn(-1, 1, 64, 8, 128, ctypes.byref(n)) == EINVAL
    assert fn(4, 0, 64, 8, 128, ctypes.byref(n)) == EINVAL
    assert fn(4, 1, 63, 8, 128, ctypes.byref(n)) == EINVAL
    assert fn(4, 1, 64, 8, 80, ctypes.byref(n)) == EUNSUP
    assert fn(4, 65, 64, 8, 128, ctypes.byref(n)) == ERANGE
    assert fn(4097, 1, 64, 8, 128, ctypes.byref(n)) == ERANGE


@pytest.mark.parametrize("kw,status", [
    (dict(pairs=None), EINVAL), (dict(count=-1), EINVAL), (dict(count=(1 << 20) + 1), ERANGE), (dict(count=0, pairs=None), OK),
    (dict(c_layers=60000, c_kv_heads=4000, c_page_size=1024), ERANGE),
])
def test_copy_refuses(kw, status):
    assert copy(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(table=None), EINVAL), (dict(ctx=None), EINVAL), (dict(keep=None), EINVAL), (dict(cols=0), EINVAL),
    (dict(ld=5), EINVAL), (dict(width=-1), EINVAL), (dict(batch=-1), EINVAL), (dict(width=1025), ERANGE),
    (dict(batch=4097), ERANGE), (dict(batch=0, table=None), OK), (dict(width=0, keep=None), OK),
    (dict(c_layers=60000, c_kv_heads=4000), ERANGE),
])
def test_compact_refuses(kw, status):
    assert compact(**kw) == status


POOL = dict(ref=FAKE, free_bits=FAKE, table=FAKE, held=FAKE, len=FAKE, status=FAKE, pages=100, page_size=16, seqs=4,
            max_pages=10)


@pytest.mark.parametrize("call", ["init", "trim", "fork", "reserve"])
@pytest.mark.parametrize("kw,status", [
    *((dict([(f, None)]), EINVAL) for f in ("ref", "free_bits", "table", "held", "len", "status")),
    *((dict([(f, 0)]), EINVAL) for f in ("pages", "seqs", "max_pages")), (dict(page_size=24), EUNSUP),
    (dict(page_size=8), EUNSUP), (dict(pages=(1 << 24) + 1), ERANGE), (dict(seqs=4097), ERANGE),
    (dict(max_pages=1 << 28), ERANGE), (dict(page_size=1024, max_pages=1 << 21), ERANGE),
])
def test_bad_pools(call, kw, status):
    d = ubw.PagePoolDesc(**(POOL | kw))
    args = [FAKE] * {"init": 0, "trim": 1, "fork": 1, "reserve": 2}[call] + [None]
    assert getattr(ubw.lib(), f"ubw_pages_{call}")(ctypes.byref(d), *args) == status


def test_pool_calls_refuse_null():
    L, p = ubw.lib(), ctypes.byref(ubw.PagePoolDesc(**POOL))
    assert L.ubw_pages_init(None, None) == EINVAL
    assert L.ubw_pages_trim(p, None, None) == EINVAL
    assert L.ubw_pages_fork(p, None, None) == EINVAL
    assert L.ubw_pages_reserve(p, None, FAKE, None) == EINVAL
    assert L.ubw_pages_reserve(p, FAKE, None, None) == EINVAL


@pytest.mark.parametrize("call,kw", [
    (rope, dict(pos=FAKE + 2)), (rope, dict(slots=FAKE + 1)), (rope, dict(freq=FAKE + 2)), (attn, dict(start=FAKE + 2)),
    (attn, dict(ctx=FAKE + 1)), (attn, dict(table=FAKE + 3)), (copy, dict(pairs=FAKE + 2)), (compact, dict(table=FAKE + 2)),
    (compact, dict(ctx=FAKE + 2)), (compact, dict(keep=FAKE + 2)),
])
def test_arrays_are_aligned(call, kw):
    assert call(**kw) == EALIGN


@pytest.mark.parametrize("field", ["ref", "free_bits", "table", "held", "len", "status"])
def test_pool_arrays_are_aligned(field):
    p = ctypes.byref(ubw.PagePoolDesc(**(POOL | {field: FAKE + 2})))
    assert ubw.lib().ubw_pages_init(p, None) == EALIGN
    assert ubw.lib().ubw_pages_trim(p, FAKE, None) == EALIGN


def test_attention_positions_stay_clear_of_32_bits():
    assert attn(cols=(1 << 26) + 1, ld_table=1 << 27) == ERANGE
