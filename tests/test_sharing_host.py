"""CPU-only checks of the page operators: their refusals before any CUDA call,
and the sequential reference held to what any right one keeps."""
import copy
import ctypes

import numpy as np
import pytest
import torch

from paged_fp8_kv_quantize_gb300 import abi
from sharing_oracle import SharedPool


def desc(**kw):
    d = abi.CacheDesc(100, 16, 8, 128, 128, 0, abi.DTYPE_FP8_E4M3, 0, 256, 256, 256, 256, 256)
    for k, v in kw.items():
        setattr(d, k, v)
    return ctypes.byref(d)


def test_a_call_takes_the_cache_as_it_is():
    """A pool that has grown, a copied cache, two calls at once: each call's
    descriptor is its own and holds what the cache is then."""
    c = abi.PagedCache(4, 16, 2, 64, device="cpu")
    cpu = c.page_tags.get_device()
    first = c._ref(cpu)._obj
    was = bytes(first)
    copied = copy.deepcopy(c)
    assert copied._ref(cpu)._obj.k_pool == copied.k_pool.data_ptr()
    shallow = copy.copy(c)
    c.P = 9
    c.k_pool, c.v_pool = (torch.zeros(9 * 2 * 16 * 64, dtype=torch.uint8) for _ in range(2))
    c.page_tags = torch.zeros(9, dtype=torch.int32)
    now = c._ref(cpu)._obj
    assert (now.num_pages, now.k_pool, now.page_tags) == (9, c.k_pool.data_ptr(), c.page_tags.data_ptr())
    assert bytes(first) == was and bytes(shallow._ref(cpu)._obj) == was
    with pytest.raises(ValueError):
        c._ref(0)  # not where the cache is


def test_copy_refusals():
    f = abi.lib.pfkv_page_copy
    assert f(None, 16, 16, None, 1, 16, None) == -1
    assert f(desc(dtype=7), 16, 16, None, 1, 16, None) == -4
    assert f(desc(k_pool=264), 16, 16, None, 1, 16, None) == -6
    assert f(desc(), 16, 16, None, -1, 16, None) == -2
    assert f(desc(), None, None, None, 0, None, None) == 0  # nothing to do, nothing launched
    for a in ((None, 16, 16), (16, None, 16), (16, 16, None)):
        assert f(desc(), a[0], a[1], None, 1, a[2], None) == -1
    # more slabs than a grid has
    assert f(desc(num_kv_heads=65536, head_dim=4096, v_head_dim=4096, page_size=1 << 20), 16, 16, None, 2, 16,
             None) == -2


def test_fork_refusals():
    f = abi.lib.pfkv_page_fork

    def call(state=256, tags=16, refs=16, c=None, par=16, chi=16, lens=16, n=1, table=16, btags=16, batch=4, mp=8,
             flags=0, st=16):
        return f(state, tags, refs, desc() if c is None else c, par, chi, lens, n, table, btags, batch, mp, flags, st,
                 None)

    assert call(n=0, par=None, chi=None, lens=None, table=None, st=None) == 0
    for k in ("state", "tags", "refs", "par", "chi", "lens", "table", "st"):
        assert call(**{k: None}) == -1, k
    assert call(btags=None, flags=abi.FLAG_TAG_CHECK) == -1
    assert call(n=-1) == call(n=65537) == call(batch=-1) == call(mp=0) == call(batch=1 << 21, mp=1 << 20) == -2
    assert call(state=272) == -6
    assert call(c=desc(page_size=0)) == -2


def test_release_refusals():
    f = abi.lib.pfkv_page_release
    assert f(256, 16, None, 0, None, None) == 0
    assert f(None, 16, 16, 1, 16, None) == f(256, None, 16, 1, 16, None) == -1
    assert f(256, 16, None, 1, 16, None) == f(256, 16, 16, 1, None, None) == -1
    assert f(256, 16, 16, -1, 16, None) == f(256, 16, 16, 1 << 30, 16, None) == -2
    assert f(272, 16, 16, 1, 16, None) == -6


def test_compact_refusals():
    f = abi.lib.pfkv_page_compact

    def call(state=256, tags=16, table=16, batch=2, mp=4, moves=3, src=16, dst=16, n=16, c=None):
        return f(state, tags, None, desc() if c is None else c, table, None, None, batch, mp, moves, src, dst, n, None)

    for k in ("state", "tags", "table", "src", "dst", "n"):
        assert call(**{k: None}) == -1, k
    assert call(batch=-1) == call(mp=0) == call(moves=-1) == call(batch=1 << 21, mp=1 << 20) == -2
    assert call(state=260) == -6
    assert call(c=desc(dtype=3)) == -4


def test_reference_keeps_the_pool_whole():
    """Random calls: the free list and the held pages part the pool, a page's
    holders are the rows that name it, every row reads what it read before a
    compaction, and a child reads its parent's tokens."""
    rng = np.random.default_rng(3)
    P, S, B, MP = 60, 4, 10, 6
    pool = SharedPool(P, np.zeros(P, dtype=np.uint32), [rng.integers(0, 256, size=(P, 2, S, 3), dtype=np.uint8)])
    table, btags, lens = np.full((B, MP), -1, np.int32), np.zeros((B, MP), np.uint32), np.zeros(B, int)

    def read(b):
        n = -(-lens[b] // S)
        return np.concatenate([pool.arrays[0][p] for p in table[b, :n]] or [np.zeros((2, 0, 3), np.uint8)], 1)[:, :lens[b]]

    for step in range(300):
        op, live, empty = rng.integers(4), np.flatnonzero(lens), np.flatnonzero(lens == 0)
        if op == 0 and empty.size:
            m = int(rng.integers(1, MP * S + 1))
            got = pool.alloc(-(-m // S))
            if got:
                b = empty[0]
                table[b, :len(got)], btags[b, :len(got)], lens[b] = got, pool.tags[got], m
        elif op == 1 and live.size and empty.size:
            par, chi = int(rng.choice(live)), int(empty[0])
            m = int(rng.integers(0, lens[par] + 1))
            if pool.fork([par], [chi], [m], table, btags, True)[0] == 0:
                lens[chi] = m
                assert np.array_equal(read(chi), read(par)[:, :m])
        elif op == 2 and live.size:
            b = int(rng.choice(live))
            assert not pool.release(table[b, : -(-lens[b] // S)].tolist()).any()
            lens[b] = 0
        elif op == 3:
            was = [read(b) for b in range(B)]
            k = int(rng.integers(0, 12))
            moves = pool.compact(table, btags, [-(-m // S) for m in lens], k)
            assert all(np.array_equal(a, read(b)) for b, a in enumerate(was))
            if len(moves) < k:
                assert not pool.held[pool.held.sum():].any()
        names = np.zeros(P, int)
        for b in range(B):
            np.add.at(names, table[b, : -(-lens[b] // S)], 1)
        assert np.array_equal(names > 0, pool.held)
        assert np.array_equal(names[pool.held] - 1, pool.refs[pool.held]) and not pool.refs[~pool.held].any()
        assert sorted(pool.stack) == np.flatnonzero(~pool.held).tolist()
        for b in range(B):
            n = -(-lens[b] // S)
            assert np.array_equal(btags[b, :n], pool.tags[table[b, :n]])
