"""CPU-only checks of the shared-prefix decode: refusals before any CUDA call,
the workspace's size, and the work line restated."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from paged_fp8_kv_quantize_gb300 import abi, build

SIZE_MAX = ctypes.c_size_t(-1).value


def desc(**kw):
    d = abi.CacheDesc(100, 16, 8, 128, 128, 0, abi.DTYPE_FP8_E4M3, 0, 256, 256, 256, 256, 256)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def call(c=None, k=None, v=None, q=256, hq=32, lens=256, table=256, tags=256, batch=4, mp=8, group=256, pages=256,
         n_groups=1, scale=1.0, flags=0, splits=64, ws=256, ws_bytes=0, out=256, out_dtype=0, st=256):
    return abi.lib.pfkv_paged_decode_attention_prefix(
        None if c is False else ctypes.byref(c or desc()), k, v, q, hq, lens, table, tags, batch, mp, group, pages,
        n_groups, scale, flags, splits, ws, ws_bytes, out, out_dtype, st, None)


def test_refusals():
    assert call(False) == -1
    for name in ("q", "lens", "table", "group", "pages", "ws", "out", "st"):
        assert call(**{name: None}) == -1, name
    assert call(k=256) == call(v=256) == -1  # both or neither
    assert call(k=264, v=256) == call(q=8) == -6
    assert call(tags=None, flags=abi.FLAG_TAG_CHECK) == -1
    assert call(hq=30) == call(batch=-1) == call(mp=0) == call(splits=0) == call(splits=257) == -2
    assert call(n_groups=-1) == call(scale=float("inf")) == call(scale=float("nan")) == -2
    assert call(batch=1 << 20, mp=1 << 21) == -2
    assert call(batch=1 << 27, hq=32) == -2  # a join block per (request, head)
    assert call(n_groups=4097) == call(batch=65536) == -3
    assert call(out_dtype=2) == call(out_dtype=-1) == -4
    assert call(desc(page_size=24)) == call(desc(page_size=272)) == -3
    lat = desc(num_kv_heads=1, head_dim=576, v_head_dim=512, kv_shared=1, scale_mode=1, page_size=64)
    assert call(lat, hq=64) == -3
    assert call() == -5  # workspace too small
    assert call(batch=0) == 0
    big = abi.lib.pfkv_prefix_workspace_bytes(ctypes.byref(desc()), 4, 32, 1, 64)
    assert call(ws_bytes=big - 1) == -5
    assert call(ws=264, ws_bytes=big) == -6
    assert call(desc(head_dim=96, v_head_dim=96), ws_bytes=1 << 40) == -3


def test_too_many_head_groups_are_refused_first():
    """More KV heads, or groups of eight query heads, than the split kernel
    takes: refused before the CUDA runtime is asked for anything."""
    assert call(desc(num_kv_heads=4097), hq=4097, ws_bytes=1 << 40) == -3
    assert call(desc(num_kv_heads=2049), hq=2049 * 9, ws_bytes=1 << 40) == -3


def test_workspace_bytes():
    f = abi.lib.pfkv_prefix_workspace_bytes
    d = desc()
    plain = abi.lib.pfkv_decode_workspace_bytes(ctypes.byref(d), 64, 32, 64)
    one = f(ctypes.byref(d), 64, 32, 1, 64)
    # a slot per range (256 at most) and per row block of a KV head, of 256 rows of 128 fp32 values and (m, l)
    rows = one - plain
    assert rows - (256 + 8 * (64 * 4 // 256 + 1)) * 256 * 520 in range(64 * 1024)
    assert f(ctypes.byref(d), 64, 32, 5, 64) > one
    assert plain < f(ctypes.byref(d), 64, 32, 0, 64) < plain + 64 * 1024
    for bad in ((64, 33, 1, 64), (64, 32, 4097, 64), (65536, 32, 1, 64), (64, 32, 1, 300)):
        assert f(ctypes.byref(d), *bad) == SIZE_MAX, bad
    assert f(None, 64, 32, 1, 64) == 0 and f(ctypes.byref(d), 64, 32, -1, 64) == 0


def test_workspace_bytes_of_what_a_call_refuses():
    f = abi.lib.pfkv_prefix_workspace_bytes
    lat = dict(num_kv_heads=1, head_dim=576, v_head_dim=512, kv_shared=1, scale_mode=1, page_size=64)
    for kw, hq in ((dict(head_dim=96, v_head_dim=96), 32), (dict(v_head_dim=64), 32), (lat, 64), (dict(page_size=24), 32),
                   (dict(page_size=272), 32), (dict(page_size=0), 32), (dict(num_kv_heads=4097), 4097),
                   (dict(num_kv_heads=2049), 2049 * 9)):
        assert f(ctypes.byref(desc(**kw)), 4, hq, 1, 64) == SIZE_MAX, kw
    assert f(ctypes.byref(desc()), 65535, 65536, 1, 64) == SIZE_MAX  # rows are counted in int
    assert f(ctypes.byref(desc(num_kv_heads=4096)), 4, 4096 * 8, 1, 64) < SIZE_MAX


ROWS, HALF, FULL = 256, 4, 7  # rows of an item; a page's cost in a block of at most half the rows, and in others


def line(groups, H, G, ctas, c0, min_units):
    """The plan restated: [(members, pages)] -> (T, R, per group (pages, first item, first unit, block costs), items)."""
    unit = item = 0
    out = []
    for n, p in groups:
        p = p if n else 0
        rows = n * G
        cost = [HALF if rows - i * ROWS <= ROWS // 2 else FULL for i in range(-(-rows // ROWS))]
        out.append((p, item, unit, cost))
        if p:
            item += H * len(cost)
            unit += H * sum(c0 + c * p for c in cost)
    return unit, 0 if unit == 0 else min(max(unit // min_units, 1), ctas), out, item


@pytest.mark.parametrize("seed", range(60))
def test_work_line_covers_every_item_once(seed):
    """Pieces of the ranges, as the planner walks them, against the slots that
    the join looks for: every page of every item once, distinct slots inside
    the workspace, and the join's range of pieces is the walk's."""
    rng = np.random.default_rng(seed)
    H, G, S = int(rng.integers(1, 9)), int(rng.integers(1, 17)), int(rng.choice([16, 48, 64, 256]))
    groups = [(int(rng.integers(0, 70)), int(rng.integers(0, 300))) for _ in range(int(rng.integers(1, 12)))]
    c0 = HALF * -(-512 // S)
    T, R, g, items = line(groups, H, G, int(rng.choice([1, 7, 152, 256])), c0, HALF * -(-256 // S))
    if T == 0:
        assert R == 0
        return
    seen, slots = {}, set()
    for k in range(R):
        u, u1 = k * T // R, (k + 1) * T // R
        while u < u1:
            lo = max(i for i, x in enumerate(g) if x[2] <= u)
            p, item0, unit0, cost = g[lo]
            full, segs = c0 + FULL * p, [c0 + c * p for c in cost]
            h, rel = divmod(u - unit0, sum(segs))
            blk = min(len(cost) - 1, rel // full)
            off = rel - blk * full
            end = min(segs[blk], off + u1 - u)
            p0, p1 = -(-max(0, off - c0) // cost[blk]), -(-max(0, end - c0) // cost[blk])
            u += end - off
            if p1 <= p0:
                continue
            slot = k + item0 + h * len(cost) + blk
            assert h < H and slot not in slots
            slots.add(slot)
            seen.setdefault((lo, h, blk), []).append((p0, p1, k, slot))
    for i, (p, item0, unit0, cost) in enumerate(g):
        for h in range(H if p else 0):
            for blk, w in enumerate(cost):
                pieces = seen.pop((i, h, blk))
                assert [x[0] for x in pieces] == [0] + [x[1] for x in pieces[:-1]] and pieces[-1][1] == p
                first = unit0 + h * sum(c0 + c * p for c in cost) + blk * (c0 + FULL * p) + c0
                k0, k1 = ((first + 1) * R - 1) // T, ((first + w * (p - 1) + 1) * R - 1) // T
                assert [x[2] for x in pieces] == list(range(k0, k1 + 1))
                assert [x[3] for x in pieces] == [k + item0 + h * len(cost) + blk for k in range(k0, k1 + 1)]
    assert not seen and max(slots) < R + items


@pytest.fixture(scope="module")
def line_faults(tmp_path_factory):
    """prefix_line.cu, built from the kernels' own headers for the host."""
    here = os.path.dirname(os.path.abspath(__file__))
    lib = str(tmp_path_factory.mktemp("prefix_line") / "prefix_line.so")
    subprocess.run([build.nvcc(), *build.ARCH, *build.FLAGS, "-I", build.CSRC, "-shared", "-o", lib,
                    os.path.join(here, "prefix_line.cu")], check=True)
    f = ctypes.CDLL(lib).prefix_line_faults
    f.restype = ctypes.c_longlong

    def call(groups, H, G, S, ctas):
        n, p = zip(*groups)
        arr = ctypes.c_int * len(groups)
        return f(arr(*n), arr(*p), len(groups), H, G, S, ctas)

    return call


@pytest.mark.parametrize("page", range(16, 257, 16))
def test_every_row_finds_its_pieces_on_short_lines(line_faults, page):
    """One group of few pages, rows on both sides of 128, 256 and 384: ranges
    are then as short as they get, and each between an item's first and last
    still has to hold a page's beginning."""
    bad = [(members, G, H, pages, ctas)
           for members, G in ((1, 1), (16, 8), (33, 4), (64, 4), (65, 4), (48, 8), (13, 33))
           for H in (1, 8) for ctas in (148, 152) for pages in (*range(1, 61), 100, 160)
           if line_faults([(members, pages)], H, G, page, ctas)]
    assert not bad, (len(bad), bad[:8])


def test_every_row_finds_its_pieces_on_mixed_lines(line_faults):
    rng = np.random.default_rng(61)
    for _ in range(400):
        groups = [(int(rng.integers(0, 90)), int(rng.integers(0, 40))) for _ in range(int(rng.integers(1, 9)))]
        args = (groups, int(rng.choice([1, 2, 8])), int(rng.integers(1, 17)), int(rng.choice(range(16, 257, 16))),
                int(rng.choice([1, 7, 148, 152, 256])))
        assert line_faults(*args) == 0, args
