"""Copies of pages in numbers that take several launches."""
import pytest

import ultra_bit_weight_uint32_amd as ubw
from test_gpu_cache import DEV, F16, gen, randn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_copies_that_take_several_launches():
    """The most pairs of one call, nearly all of them skipped: 4 pieces a page in 5 layers make 838860 pairs a
    launch. Valid pairs lie at the ends of both launches."""
    g = gen(1)
    layers, pages, kv, page, dim = 5, 9, 8, 16, 256
    k, v = (randn((layers, pages, kv, page, dim), F16, g) for _ in "kv")
    cache = ubw.KVCache(k, v)
    count, per = 1 << 20, ((1 << 24) - 1) // (4 * layers)
    assert count > per
    pairs = torch.full((count, 2), -1, dtype=torch.int32, device=DEV)
    want = [k.clone(), v.clone()]
    for at, (a, b) in {0: (0, 5), per - 1: (1, 6), per: (2, 7), count - 1: (3, 8)}.items():
        pairs[at, 0], pairs[at, 1] = a, b
        for w in want:
            w[:, b] = w[:, a]
    ubw.cache_copy_pages(cache, pairs)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
