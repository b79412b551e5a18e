"""Page copy, fork, release and compact on the GPU against the sequential
reference: every table entry, tag, holder count, status, the free list and
every byte of the pools after each call."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev_i32
from paged_fp8_kv_quantize_gb300 import abi
from sharing_oracle import SharedPool

pytestmark = pytest.mark.gpu

# kind: (page size, heads, head dim, v head dim, shared stream, dtype, scale mode).  "odd" has pages of 24 and 40
# bytes per row and three slots (8-byte vectors, pages that start off 16 bytes)
KINDS = {
    "fp8": (16, 2, 128, 128, False, abi.DTYPE_FP8_E4M3, abi.SCALE_PER_HEAD),
    "fp8_token": (16, 3, 64, 64, False, abi.DTYPE_FP8_E4M3, abi.SCALE_PER_TOKEN),
    "bf16": (64, 2, 64, 64, False, abi.DTYPE_BF16, abi.SCALE_PER_HEAD),
    "latent": (64, 1, 576, 512, True, abi.DTYPE_FP8_E4M3, abi.SCALE_PER_TOKEN),
    "odd": (3, 5, 40, 40, False, abi.DTYPE_FP8_E4M3, abi.SCALE_PER_TOKEN),
    "one_slot": (1, 1, 8, 8, False, abi.DTYPE_BF16, abi.SCALE_PER_HEAD),
}


def u32(t):
    return t.cpu().numpy().view(np.uint32)


class Pair:
    """The same pool on the GPU and in the reference."""

    def __init__(self, kind, P, B, MP, seed):
        S, H, D, Dv, shared, dtype, mode = KINDS[kind]
        rng = np.random.default_rng(seed)
        self.S, self.P, self.rng = S, P, rng
        self.cache = abi.PagedCache(P, S, H, D, Dv, shared, dtype, mode)
        self.gpu_arrays = [(self.cache.k_pool, D), (self.cache.v_pool, Dv)]
        if mode == abi.SCALE_PER_TOKEN:
            self.gpu_arrays += [(self.cache.k_scale, 1), (self.cache.v_scale, 1)]
        self.gpu_arrays = [(t, d) for t, d in self.gpu_arrays if t is not None]
        arrays = []
        for t, d in self.gpu_arrays:
            raw = rng.integers(0, 256, size=t.numel() * t.element_size(), dtype=np.uint8)
            t.view(torch.uint8).copy_(torch.from_numpy(raw))
            arrays.append(raw.reshape(P, H, S, d * t.element_size()))
        tags = rng.integers(0, 1 << 32, size=P, dtype=np.uint64).astype(np.uint32)
        tags[:2] = 0xFFFFFFFF  # wraps on the next hand-out
        self.cache.page_tags.copy_(dev_i32(tags))
        self.alloc = abi.PageAllocator(P)
        self.ref = SharedPool(P, tags, arrays)
        self.table = np.full((B, MP), -1, dtype=np.int32)
        self.btags = np.zeros((B, MP), dtype=np.uint32)
        self.lens = np.zeros(B, dtype=np.int32)
        self.upload()

    def upload(self):
        self.gtable, self.gtags = dev_i32(self.table), dev_i32(self.btags)

    def fill_row(self, b, n_tokens):
        """A row of its own pages."""
        need = -(-n_tokens // self.S)
        pages, tags, st = self.alloc.alloc(need, self.cache.page_tags)
        got = self.ref.alloc(need)
        if got is None:
            assert u32(st)[0] == abi.ST_NO_PAGES
            return
        assert pages.cpu().tolist() == got
        self.table[b, :need], self.btags[b, :need] = got, self.ref.tags[got]
        self.lens[b] = n_tokens
        self.upload()

    def check(self, where):
        torch.cuda.synchronize()
        assert np.array_equal(self.gtable.cpu().numpy(), self.table), where
        assert np.array_equal(u32(self.gtags), self.btags), where
        assert np.array_equal(u32(self.cache.page_tags), self.ref.tags), where
        assert np.array_equal(self.alloc.refs.cpu().numpy(), self.ref.refs), where
        assert self.alloc.free_count() == len(self.ref.stack), where
        assert self.alloc.free_list().cpu().tolist() == self.ref.stack, where
        for (t, _), a in zip(self.gpu_arrays, self.ref.arrays):
            assert np.array_equal(t.view(torch.uint8).cpu().numpy(), a.reshape(-1)), where

    def fork(self, parents, children, lens, flags=abi.FLAG_TAG_CHECK):
        st = self.alloc.fork(self.cache, dev_i32(np.array(parents)), dev_i32(np.array(children)),
                             dev_i32(np.array(lens)), self.gtable, self.gtags, flags=flags)
        want = self.ref.fork(list(parents), list(children), list(lens), self.table, self.btags, bool(flags))
        assert np.array_equal(u32(st), want), (u32(st), want)
        for c, m, s in zip(children, lens, want):
            if s == 0:
                self.lens[c] = m
        return want

    def release(self, pages):
        st = self.alloc.release(dev_i32(np.array(pages, dtype=np.int32)))
        want = self.ref.release(pages)
        assert np.array_equal(u32(st), want)
        return want

    def compact(self, used=None, max_moves=None, tags=True):
        src, dst, n = self.alloc.compact(self.cache, self.gtable, self.gtags if tags else None,
                                         used=None if used is None else dev_i32(np.array(used)),
                                         max_moves=max_moves)
        moves = self.ref.compact(self.table, self.btags if tags else None, used,
                                 self.P if max_moves is None else max_moves)
        torch.cuda.synchronize()
        assert int(n.item()) == len(moves)
        got = list(zip(src.cpu().tolist()[:len(moves)], dst.cpu().tolist()[:len(moves)]))
        assert got == moves
        return moves


@pytest.mark.parametrize("kind", list(KINDS))
def test_copy_matches_reference(kind):
    p = Pair(kind, 41, 1, 1, 1)
    ids = p.rng.permutation(41)
    src, dst = ids[:15].astype(np.int32), ids[15:30].astype(np.int32)
    slots = p.rng.integers(0, p.S + 1, size=15).astype(np.int32)
    src[3], dst[5], slots[7], slots[8], dst[9] = 41, -1, p.S + 1, -1, src[9]  # refused, and a page onto itself
    slots[0], slots[1] = 0, p.S
    for sl in (slots, None):
        st = abi.page_copy(p.cache, dev_i32(src), dev_i32(dst), None if sl is None else dev_i32(sl))
        assert np.array_equal(u32(st), p.ref.copy(src, dst, sl))
        p.check("slots" if sl is not None else "whole pages")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert abi.page_copy(p.cache, none, none).numel() == 0


@pytest.mark.parametrize("kind", list(KINDS))
def test_fork_release_compact_sequences(kind):
    """Random calls one after another, with lists that hold refused entries:
    rows and pages out of range, lengths past the table, repeated children,
    a child that is a parent, stale tags, pages given back too often."""
    B, MP = 14, 9
    p = Pair(kind, 83, B, MP, 2)
    for b in range(4):
        p.fill_row(b, int(p.rng.integers(1, MP * p.S + 1)))
    p.check("start")
    seen = np.zeros(4, dtype=int)
    for step in range(50):
        op = int(p.rng.integers(4))
        live = np.flatnonzero(p.lens > 0)
        if op == 0 and live.size:
            n = int(p.rng.integers(1, 5))
            empty = np.flatnonzero(p.lens == 0)
            par = p.rng.choice(live, size=n)
            chi = p.rng.choice(empty, size=n, replace=empty.size < n) if empty.size else par
            m = np.array([p.rng.integers(0, p.lens[b] + 1) for b in par])
            bad = p.rng.random(n)
            par = np.where(bad < 0.05, B, par)
            chi = np.where((bad > 0.05) & (bad < 0.1), -1, chi)
            m = np.where((bad > 0.1) & (bad < 0.15), MP * p.S + 1, m)
            if step % 7 == 0:  # a mapping from before a reallocation
                p.btags[par[0] % B, 0] ^= np.uint32(1)
                p.upload()
            st = p.fork(par.tolist(), chi.tolist(), m.tolist(), abi.FLAG_TAG_CHECK if step % 3 else 0)
            seen[0] += int((st == 0).sum())
        elif op == 1 and live.size:
            b = int(p.rng.choice(live))
            pages = p.table[b, : -(-int(p.lens[b]) // p.S)].tolist()
            pages += [-1, p.P][: int(p.rng.integers(3))] + ([pages[0]] if p.rng.random() < 0.2 else [])
            # an over-release takes the page from its other holders, as the reference does
            p.release(pages)
            p.table[b], p.lens[b] = -1, 0
            p.upload()
            seen[1] += 1
        elif op == 2:
            used = [-(-int(m) // p.S) for m in p.lens]
            k = int(p.rng.integers(3))
            moves = p.compact(used=used if k else None, max_moves=int(p.rng.integers(0, 9)) if k == 2 else None)
            seen[2] += len(moves)
        else:
            empty = np.flatnonzero(p.lens == 0)
            if empty.size:
                p.fill_row(int(empty[0]), int(p.rng.integers(1, MP * p.S + 1)))
            seen[3] += 1
        p.check((step, op))
    assert (seen > 0).all(), seen


def test_fork_refusals_and_exhaustion():
    p = Pair("fp8", 12, 8, 4, 3)
    p.fill_row(0, 4 * 16)
    p.fill_row(1, 40)
    free0 = p.alloc.free_count()
    # each refusal alone; sound entries of the same call are done
    st = p.fork([0, 0, 8, 0, 1, 1, 1], [2, 2, 3, 0, 1, 4, -1], [64, 20, 3, 10, 10, 4 * 16 + 1, 8])
    assert st.tolist() == [0, 64, 128, 64, 64, 4, 128]
    p.check("refusals")
    assert p.alloc.free_count() == free0  # 64 tokens are whole pages: nothing taken
    # a page of the parent that is not handed out; a page id outside the pool
    p.table[5, :2] = [11, 99]
    p.upload()
    assert p.fork([5, 5], [6, 7], [16, 32], flags=0).tolist() == [32, 32 | 2]
    p.check("foreign pages")
    # five free pages, six wanted: none is taken, whole-page forks of the call are not done either
    assert p.alloc.free_count() == 5
    p2 = Pair("fp8", 9, 8, 4, 4)
    p2.fill_row(0, 50)
    st = p2.fork([0] * 7, [1, 2, 3, 4, 5, 6, 7], [50, 17, 1, 15, 16, 33, 34])
    assert (st == abi.ST_NO_PAGES).all()
    p2.check("exhausted")
    assert (p2.fork([0] * 3, [1, 2, 3], [50, 0, 48]) == 0).all()
    p2.check("after")


def test_release_counts_holders():
    p = Pair("fp8", 20, 6, 3, 5)
    p.fill_row(0, 48)
    assert (p.fork([0, 0, 0], [1, 2, 3], [48, 48, 32]) == 0).all()
    a, b, c = p.table[0, :3].tolist()
    assert p.alloc.refs.cpu().numpy()[[a, b, c]].tolist() == [3, 3, 2]
    # four holders of a: two in this list, the page stays
    assert (p.release([a, c, a]) == 0).all()
    p.check("still held")
    # c: two holders left, listed three times, so it goes back at once; b: four, listed four times
    st = p.release([c, b, b, c, c, b, b])
    assert st.tolist() == [0, 0, 0, 32, 32, 0, 0]
    p.check("given back in list order")
    assert p.alloc.free_list().cpu().tolist()[-2:] == [c, b]
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert p.alloc.release(none).numel() == 0


@pytest.mark.parametrize("n_rows,forks", [(3, 40), (2, 1000)])
def test_release_of_long_lists(n_rows, forks):
    """Lists above and below the one-block limit: every child row of a wide
    fork given back at once, its pages shared by all of them."""
    MP = 11
    p = Pair("one_slot", 600 + 2 * forks, n_rows + forks, MP, 6)
    for b in range(n_rows):
        p.fill_row(b, MP - b)
    par = [i % n_rows for i in range(forks)]
    chi = list(range(n_rows, n_rows + forks))
    assert (p.fork(par, chi, [int(p.lens[b]) for b in par]) == 0).all()
    p.check("forked")
    pages = [int(q) for c in chi for q in p.table[c, : p.lens[c]]]
    half = pages[: len(pages) // 2] + [-7]
    p.release(half)
    p.check("half")
    p.release(pages[len(pages) // 2:])
    p.check("all children")
    assert not p.alloc.refs.any()
    # every parent's page twice: the second time nobody holds it
    again = [int(q) for b in range(n_rows) for q in p.table[b, : p.lens[b]]] * 2
    st = p.release(again)
    assert st.tolist() == [0] * (len(again) // 2) + [32] * (len(again) // 2)
    p.check("parents")
    # one page listed thousands of times
    p.release([again[0]] * 5000)
    p.check("never held")


@pytest.mark.parametrize("repeat", [1, 900])
def test_pages_listed_more_often_than_held(repeat):
    """Short and long lists (one block, several): a page goes back at its first
    listing, the rest of its listings are refused, and others are not touched."""
    p = Pair("one_slot", 64, 6, 30, 8)
    p.fill_row(0, 12)
    p.fill_row(1, 5)
    p.fork([0, 0, 1], [2, 3, 4], [12, 7, 5])  # three holders of seven pages, two of ten
    a, b, c = p.table[0, 0], p.table[0, 9], p.table[1, 2]
    pages = [b, a, c, a, b, a, 63, a, b, c, -1] + [a, 64, b] * repeat + [p.table[0, 1]]
    st = p.release([int(x) for x in pages])
    assert (st == 0).sum() == 5 and st[0] == st[1] == st[2] == st[9] == st[-1] == 0
    p.check("released")
    p.release([int(x) for x in pages] + [int(p.table[0, 1])] * 2 * repeat)
    p.check("again")


def test_release_without_sharing_is_free():
    rng = np.random.default_rng(7)
    P = 9000
    tags = torch.zeros(P, dtype=torch.int32, device="cuda")
    a, b = abi.PageAllocator(P), abi.PageAllocator(P)
    for x in (a, b):
        x.alloc(8000, tags)
    for n in (17, 4096, 6000):
        ids = dev_i32(rng.integers(-2, P + 2, size=n).astype(np.int32))
        assert torch.equal(a.free(ids), b.release(ids))
        assert torch.equal(a.free_list(), b.free_list())
    assert not b.refs.any()


@pytest.mark.parametrize("P", [3000, 20000])  # one block plans the moves; many do
def test_compact_bounds_and_stale_rows(P):
    p = Pair("one_slot" if P > 3000 else "fp8_token", P, 5, 400, 8)
    others = p.ref.alloc(P // 3)  # pages of other owners among the rows', two in three given back
    assert p.alloc.alloc(P // 3, p.cache.page_tags)[0].tolist() == others
    for b in range(5):
        p.fill_row(b, 220 * p.S if P == 3000 else 380 * p.S)
        assert p.lens[b]
    p.release(p.rng.permutation(others)[: 2 * len(others) // 3].tolist())
    for b in (0, 2):
        p.release(p.table[b, :220 if P == 3000 else 380].tolist())
        p.table[b] = -1
    p.table[4, 390:] = p.table[4, 210:220]  # past the live entries: left as they were
    p.btags[4, 5] ^= np.uint32(1)  # a stale mapping stays stale
    p.upload()
    used = [0, *([220] if P == 3000 else [380]), 0, *([220, 220] if P == 3000 else [380, 380])]
    before = p.table.copy()
    assert p.compact(used=used, max_moves=0) == []
    assert len(p.compact(used=used, max_moves=33)) == 33
    p.check("33 moves")
    moves = p.compact(used=used)
    p.check("the rest")
    assert moves and p.table[4, 5] == before[4, 5] and np.array_equal(p.table[4, 390:], before[4, 390:])
    assert p.compact(used=used) == []
    p.check("nothing left")


@pytest.mark.parametrize("P", [1, 2, 15, 16, 17, 1024, 16384, 16385])
def test_compact_pool_sizes(P):
    p = Pair("one_slot", P, 3, P, 14)
    p.fill_row(0, max(1, P // 2))
    p.fill_row(1, P - max(1, P // 2) - P // 5)
    if P > 1:
        gone = p.rng.permutation(p.table[0, : p.lens[0]])[: P // 3].tolist()
        p.release(gone)
        p.table[0][np.isin(p.table[0], gone)] = -1
        p.upload()
    p.compact(max_moves=P // 9)
    p.check("some")
    p.compact()
    p.check("all")


def test_compact_empty_full_and_without_tags():
    # an empty pool and a full one
    for n in (0, 50):
        q = Pair("one_slot", 50, 1, 50, 9)
        if n:
            q.fill_row(0, n)
        assert q.compact() == []
        q.check(n)
    q = Pair("bf16", 30, 2, 15, 10)
    q.fill_row(0, 10 * 64)
    q.fill_row(1, 10 * 64)
    q.release(q.table[0, :10].tolist())
    q.table[0] = -1
    q.upload()
    assert len(q.compact(tags=False)) == 10
    q.check("without tags")


def test_another_pools_allocator_is_refused():
    p = Pair("fp8", 20, 3, 4, 11)
    p.fill_row(0, 40)
    p.alloc.release(dev_i32(np.array([0])))
    p.ref.release([0])
    other = abi.PageAllocator(21)
    st = other.fork(p.cache, dev_i32(np.array([0])), dev_i32(np.array([1])), dev_i32(np.array([20])), p.gtable,
                    p.gtags)
    assert u32(st)[0] & abi.ST_PAGE_OOB
    _, _, n = other.compact(p.cache, p.gtable, p.gtags)
    assert int(n.item()) == 0 and other.free_count() == 21
    p.check("untouched")


def test_fork_release_compact_in_a_captured_graph():
    """A fork and the release of its rows, captured and replayed: every replay
    takes the pages anew."""
    p = Pair("fp8", 40, 6, 5, 12)
    p.fill_row(0, 70)
    par, chi, m = (dev_i32(np.array(v)) for v in ([0, 0], [1, 2], [70, 33]))
    at = torch.tensor([1 * 5 + k for k in range(5)] + [2 * 5 + k for k in range(3)], device="cuda")
    st = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    rel = torch.full((8,), -1, dtype=torch.int32, device="cuda")
    # once outside the graph, as a program warms up before it captures
    p.fork([0, 0], [1, 2], [70, 33])
    p.release(p.table.reshape(-1)[at.cpu().numpy()].tolist())
    p.check("warm-up")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        p.alloc.fork(p.cache, par, chi, m, p.gtable, p.gtags, flags=abi.FLAG_TAG_CHECK, fork_status=st)
        p.alloc.release(p.gtable.view(-1)[at], page_status=rel)
    for _ in range(3):
        g.replay()
        assert (p.ref.fork([0, 0], [1, 2], [70, 33], p.table, p.btags, True) == 0).all()
        assert (p.ref.release(p.table.reshape(-1)[at.cpu().numpy()].tolist()) == 0).all()
        p.check("replay")
        assert not st.any() and not rel.any()


def test_wrong_arguments_are_refused():
    p = Pair("fp8", 8, 2, 2, 13)
    i = dev_i32(np.array([0, 1]))
    with pytest.raises(ValueError):
        abi.page_copy(p.cache, i, dev_i32(np.array([1])))
    with pytest.raises(ValueError):
        abi.page_copy(p.cache, i.long(), i)
    with pytest.raises(ValueError):
        p.alloc.fork(p.cache, i, i, dev_i32(np.array([1])), p.gtable, p.gtags)
    with pytest.raises(ValueError):
        p.alloc.compact(p.cache, p.gtable, p.gtags, used=dev_i32(np.array([1, 1, 1])))
    with pytest.raises(ValueError):
        p.alloc.release(torch.zeros(2, dtype=torch.int32))
    with pytest.raises(abi.PfkvError):
        p.alloc.fork(p.cache, i, i, i, p.gtable, None, flags=abi.FLAG_TAG_CHECK)
    with pytest.raises(abi.PfkvError):
        p.alloc.compact(p.cache, p.gtable, p.gtags, max_moves=-1)
