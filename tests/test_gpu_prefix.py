"""Shared-prefix decode attention against the fp64 oracle, which knows nothing
of groups: every request by itself over its whole table."""
import math

import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import dev_bf16, dev_i32
from paged_fp8_kv_quantize_gb300 import abi, synth
from prefix_helpers import BF16, FP8, FP8_TOKEN, PrefixCase

pytestmark = pytest.mark.gpu

OUT = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("out", list(OUT))
@pytest.mark.parametrize("cache", [FP8, FP8_TOKEN, BF16])
@pytest.mark.parametrize("dim", [64, 128])
def test_types(cache, dim, out):
    """Members scattered over the batch, a request of its own, a group without
    a prefix, one without members, one with a single request."""
    c = PrefixCase(1, [0, 2, -1, 0, 1, 0, 4, 2], [5, 0, 11, 3, 2], [1, 17, 40, 16, 33, 90, 5, 300], q_heads=8,
                   kv_heads=2, dim=dim, page=16, cache=cache)
    c.assert_matches(OUT[out], abi.FLAG_TAG_CHECK)


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (3, 3), (8, 4), (9, 3), (20, 4), (14, 2), (16, 2), (32, 2), (24, 1)])
def test_head_layouts(q_heads, kv_heads):
    c = PrefixCase(2, [0] * 7 + [1] * 3, [9, 4], [3, 50, 1, 16, 15, 17, 200, 8, 31, 64], q_heads=q_heads,
                   kv_heads=kv_heads, dim=64, page=16)
    c.assert_matches()


@pytest.mark.parametrize("page", [16, 48, 64, 112, 256])
@pytest.mark.parametrize("pages", [1, 3, 20])
def test_page_sizes(page, pages):
    c = PrefixCase(3, [0, 0, 1, 0], [pages, 1], [1, page, page + 1, 2 * page - 1], q_heads=8, kv_heads=2, dim=128,
                   page=page, cache=FP8_TOKEN)
    c.assert_matches(flags=abi.FLAG_TAG_CHECK)


@pytest.mark.parametrize("page", [16, 48, 112, 240, 256])
@pytest.mark.parametrize("members", [3, 36, 75])
@pytest.mark.parametrize("pages", [2, 9])
def test_page_sizes_of_larger_groups(page, members, pages):
    """12, 144 and 300 rows: both halves of an item on their own tokens, on the
    same ones, and two items.  The workspace holds NaN, so that a partial
    result that nobody wrote shows."""
    c = PrefixCase(23, [0] * members, [pages], [1 + 37 * i % (2 * page) for i in range(members)], q_heads=8,
                   kv_heads=2, dim=64, page=page)
    ws = torch.full((abi.prefix_workspace_bytes(c.device(), members, 8, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    c.assert_matches(workspace=ws)


def test_few_large_pages_of_many_heads():
    """Ranges as short as they get, page 256: a group of 256 rows, eight KV heads."""
    c = PrefixCase(24, [0] * 64, [9], [1 + 5 * i for i in range(64)], q_heads=32, kv_heads=8, dim=64, page=256)
    ws = torch.full((abi.prefix_workspace_bytes(c.device(), 64, 32, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    c.assert_matches(workspace=ws)


@pytest.mark.parametrize("members", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 130])
def test_row_counts(members):
    """Rows on both sides of the row block's and the instruction's edges."""
    c = PrefixCase(4, [0] * members, [13], [1 + 7 * (i % 5) for i in range(members)], q_heads=16, kv_heads=2, dim=64,
                   page=16)
    c.assert_matches()


@pytest.mark.parametrize("cache,out", [(FP8, "fp32"), (FP8, "bf16"), (FP8_TOKEN, "fp32"), (BF16, "fp32"), (BF16, "bf16")])
def test_long_prefix_in_many_pieces(cache, out):
    """A prefix that every CTA takes a part of; a peaked softmax."""
    c = PrefixCase(5, [0] * 20 + [1] * 5, [700, 90], [1 + 37 * i for i in range(25)], q_heads=16, kv_heads=2, dim=128,
                   page=16, cache=cache, spread=4.0)
    c.assert_matches(OUT[out])


@pytest.mark.parametrize("max_splits", [1, 2, 3, 256])
def test_split_bounds(max_splits):
    c = PrefixCase(6, [0, 0, -1, 1], [40, 7], [1, 2000, 900, 17], q_heads=8, kv_heads=2, dim=64, page=16)
    c.assert_matches(max_splits=max_splits)


def test_nothing_shared_and_everything_shared():
    c = PrefixCase(7, [-1] * 5, [], [1, 16, 100, 33, 7], q_heads=8, kv_heads=2, dim=64, page=16)
    c.assert_matches(where="no groups")
    c = PrefixCase(8, [0] * 5, [4], [0] * 5, q_heads=8, kv_heads=2, dim=64, page=16)
    c.assert_matches(where="no own tokens")
    c = PrefixCase(9, [0], [1], [0], q_heads=1, kv_heads=1, dim=128, page=16, cache=BF16)
    c.assert_matches(where="one request, one page")
    none = abi.paged_decode_attention_prefix(
        c.device(), torch.empty(0, 1, 128, dtype=torch.bfloat16, device="cuda"), dev_i32(np.zeros(0, np.int32)),
        dev_i32(np.zeros((0, 3), np.int32)), None, dev_i32(np.zeros(0, np.int32)), dev_i32(c.pages), 0.1)
    assert none[0].shape == (0, 1, 128)


def test_more_groups_than_a_warp_holds():
    n = 150
    rng = np.random.default_rng(10)
    c = PrefixCase(10, rng.integers(-1, n, size=120).tolist(), rng.integers(0, 9, size=n).tolist(),
                   rng.integers(1, 40, size=120).tolist(), q_heads=4, kv_heads=2, dim=64, page=16)
    c.assert_matches(flags=abi.FLAG_TAG_CHECK)


def test_same_as_the_plain_decode():
    c = PrefixCase(11, [0] * 9 + [-1], [30], [20 * i + 1 for i in range(10)], q_heads=32, kv_heads=8, dim=128, page=16)
    got = c.assert_matches()
    plain, st = abi.paged_decode_attention(c.gpu, dev_bf16(c.q), dev_i32(c.lens), dev_i32(c.table), dev_i32(c.tags),
                                           c.tau)
    out, _, mag = c.want()
    assert ((got - plain).abs().cpu().numpy() <= 2 * c.tolerance(out, mag, torch.float32)).all()
    again, _ = c.call()
    assert torch.equal(got, again)  # the same call gives the same bits


def test_faults_stay_with_their_requests():
    group = [0, 0, 0, 0, 0, 1, 1, 1, 2, 2, -2, 3, 0, -1, 9]
    c = PrefixCase(12, [g if -1 <= g < 3 else -1 for g in group], [6, 4, 5], [20 + i for i in range(15)], q_heads=8,
                   kv_heads=2, dim=64, page=16)
    c.group[:] = group
    c.pages = np.array([6, 4, 5, 99], np.int32)
    want = np.zeros(15, np.uint32)
    c.tags[1, 2] ^= 1  # a stale mapping inside the prefix
    want[1] = abi.ST_STALE_TAG
    c.table[2, 3] = c.table[6, 2]  # another page than its group's
    c.tags[2, 3] = c.tags[6, 2]
    want[2] = abi.ST_PREFIX_DIFFERS
    c.table[3, 0] = c.P  # outside the pool
    want[3] = abi.ST_PAGE_OOB | abi.ST_PREFIX_DIFFERS
    c.lens[4] = 6 * 16 - 1  # ends inside the prefix
    want[4] = abi.ST_BAD_LEN
    c.tags[5, 0] ^= 1  # the group's first request itself
    want[5] = abi.ST_STALE_TAG
    c.table[7, 4] = -1  # an own page
    want[7] = abi.ST_PAGE_OOB
    c.lens[8] = 0
    want[8] = abi.ST_BAD_LEN
    want[10] = abi.ST_BAD_GROUP
    want[11] = abi.ST_BAD_GROUP  # 99 pages do not fit the table
    c.tags[12, 6] ^= 1  # an own page's stale mapping
    want[12] = abi.ST_STALE_TAG
    want[14] = abi.ST_BAD_GROUP
    got, st = c.call(flags=abi.FLAG_TAG_CHECK)
    assert st.cpu().numpy().view(np.uint32).tolist() == want.tolist()
    assert not got[torch.from_numpy(want != 0).cuda()].any()
    fine = np.flatnonzero(want == 0)
    out, _, mag = c.want()
    tol = c.tolerance(out, mag, torch.float32)
    assert (np.abs(got.cpu().numpy() - out)[fine] <= tol[fine]).all()
    # the same tables without the tag check
    _, st = c.call()
    want[want == abi.ST_STALE_TAG] = 0
    assert st.cpu().numpy().view(np.uint32).tolist() == want.tolist()


@pytest.mark.parametrize("members", [9, 40])
def test_unused_rows_of_a_padded_batch(members):
    """Rows without a request keep their group with a length of 0 or one that
    ends inside the prefix: the group's pages are those of the first row that
    has them, and the others take no part."""
    c = PrefixCase(21, [0] * members + [1, 1], [20, 3], [7 * i + 1 for i in range(members + 2)], q_heads=16,
                   kv_heads=2, dim=64, page=16)
    unused = [0, 3, members - 1, members]
    c.lens[unused] = [0, -1, 20 * 16 - 1, 0]
    c.table[unused] = -1
    got, st = c.call(flags=abi.FLAG_TAG_CHECK)
    want = np.where(np.isin(np.arange(members + 2), unused), abi.ST_BAD_LEN, 0)
    assert st.tolist() == want.tolist() and not got[unused].any()
    out, _, mag = c.want()
    used = np.flatnonzero(want == 0)
    assert (np.abs(got.cpu().numpy() - out) <= c.tolerance(out, mag, torch.float32))[used].all()
    c.lens[:] = 0  # a batch of nothing
    got, st = c.call()
    assert (st == abi.ST_BAD_LEN).all() and not got.any()


def test_first_request_with_a_page_outside_the_pool():
    """The page is never fetched; the group's other requests have another page there."""
    c = PrefixCase(13, [0, 0, 0, -1], [3], [5, 6, 7, 8], q_heads=4, kv_heads=1, dim=64, page=16)
    for bad in (-7, c.P, 2**31 - 1):
        keep = c.table[0, 1]
        c.table[0, 1] = bad
        got, st = c.call()
        assert st.tolist() == [abi.ST_PAGE_OOB] + [abi.ST_PREFIX_DIFFERS] * 2 + [0]
        assert not got[:3].any() and got[3].any()
        c.table[:3, 1] = bad  # all of them
        _, st = c.call()
        assert st.tolist() == [abi.ST_PAGE_OOB] * 3 + [0]
        c.table[:3, 1] = keep


def test_first_request_with_another_page():
    """A wrong entry in the group's first row refuses the others, and only that
    group; a stale tag there refuses nobody else; in a later row it is that
    row's alone."""
    c = PrefixCase(27, [1, 0, 0, 0, 1, -1], [4, 2], [5, 6, 7, 8, 9, 10], q_heads=4, kv_heads=1, dim=64, page=16)
    spare = int(np.setdiff1d(np.arange(c.P), c.table)[0])
    right, diff = c.table[1, 2], abi.ST_PREFIX_DIFFERS

    def status(row, page, tag=0):
        c.table[row, 2] = page
        c.tags[row, 2] = c.page_tags[page] ^ np.uint32(tag)
        got, st = c.call(flags=abi.FLAG_TAG_CHECK)
        out, _, mag = c.want()
        tol = c.tolerance(out, mag, torch.float32)
        fine = np.flatnonzero(st.cpu().numpy() == 0)
        assert (np.abs(got.cpu().numpy() - out) <= tol)[fine].all() and not got[st != 0].any()
        c.table[row, 2], c.tags[row, 2] = right, c.page_tags[right]
        return st.tolist()

    assert status(1, spare) == [0, 0, diff, diff, 0, 0]
    assert status(1, right, 1) == [0, abi.ST_STALE_TAG, 0, 0, 0, 0]
    assert status(2, spare) == [0, 0, diff, 0, 0, 0]
    assert status(2, right) == [0] * 6


@pytest.mark.parametrize("cache,page", [(FP8, 16), (FP8_TOKEN, 32), (BF16, 16)])
def test_step_appends_then_attends(cache, page):
    c = PrefixCase(14, [0, 0, -1, 1, 0], [3, 2], [1, page, 2 * page + 3, 40, 0], q_heads=8, kv_heads=2, dim=128,
                   page=page, cache=cache)
    k = synth.bf16_bits(c.rng.standard_normal((5, 2, 128), dtype=np.float32))
    v = synth.bf16_bits(c.rng.standard_normal((5, 2, 128), dtype=np.float32))
    c.device()
    got, st = c.call(flags=abi.FLAG_TAG_CHECK, k_new=dev_bf16(k), v_new=dev_bf16(v))
    assert st.tolist() == [0, 0, 0, 0, abi.ST_BAD_LEN]  # the last one's new token would fall inside the prefix
    keep = c.lens[4]
    c.lens[4] = 0
    pos = np.maximum(c.lens - 1, 0)
    pos[4] = -1
    c.ref.append(k, v, pos, c.table, c.tags, flags=abi.FLAG_TAG_CHECK)
    assert np.array_equal(c.gpu.k_pool.view(torch.uint8).cpu().numpy(), c.ref.k_pool.view(np.uint8))
    assert np.array_equal(c.gpu.v_pool.view(torch.uint8).cpu().numpy(), c.ref.v_pool.view(np.uint8))
    if cache == FP8_TOKEN:
        assert np.array_equal(c.gpu.k_scale.cpu().numpy(), c.ref.k_scale)
        assert np.array_equal(c.gpu.v_scale.cpu().numpy(), c.ref.v_scale)
    out, _, mag = c.want(abi.FLAG_TAG_CHECK)
    c.assert_close(got, out, mag, torch.float32)
    assert not got[4].any()
    c.lens[4] = keep


def test_slots_past_the_length_do_not_matter():
    """Unwritten slots of a request's last page hold anything, NaN among it."""
    for cache in (FP8, FP8_TOKEN, BF16):
        c = PrefixCase(15, [0, 0, -1, 0], [2], [1, 9, 21, 15], q_heads=8, kv_heads=2, dim=64, page=16, cache=cache)
        ref = c.call()[0].clone()
        for b in range(4):
            n = int(c.lens[b])
            p, s = int(c.table[b, (n - 1) // 16]), (n - 1) % 16 + 1
            for x in (c.gpu.k_rows(), c.gpu.v_rows()):
                if cache == BF16:
                    x[p, :, s:] = float("nan")
                else:
                    x[p, :, s:] = 0x7F
            if cache == FP8_TOKEN:
                for x in (c.gpu.k_scale, c.gpu.v_scale):
                    x.view(c.P, 2, 16)[p, :, s:] = float("inf")
        assert torch.equal(c.call()[0], ref), cache


def test_captured_and_replayed_with_other_lengths():
    c = PrefixCase(16, [0, 1, 0, -1, 1, 0], [8, 3], [1, 2, 3, 4, 5, 6], q_heads=8, kv_heads=2, dim=64, page=16, room=60)
    c.device()
    a = c.args()
    ws = torch.empty(abi.prefix_workspace_bytes(c.gpu, 6, 8, 2), dtype=torch.uint8, device="cuda")
    out = torch.empty(6, 8, 64, device="cuda")
    st = torch.empty(6, dtype=torch.int32, device="cuda")
    c.call(**a, workspace=ws, out=out, status=st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(**a, workspace=ws, out=out, status=st)
    for k in (0, 13, 50):
        c.lens = (c.lens + k).astype(np.int32)
        a["seq_lens"].copy_(dev_i32(c.lens))
        ws.fill_(0xEE)  # scratch between calls
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        want, _, mag = c.want()
        assert not st.any()
        c.assert_close(out, want, mag, torch.float32, k)
        c.lens = (c.lens - k).astype(np.int32)


def test_on_a_side_stream_beside_another_call():
    """Two calls on two streams with workspaces of their own."""
    cs = [PrefixCase(17 + i, [0] * 12, [60 + 9 * i], [5 * j + 1 for j in range(12)], q_heads=16, kv_heads=4, dim=128,
                     page=16) for i in range(2)]
    want = [c.call()[0].clone() for c in cs]
    args = [c.args() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (c, s) in enumerate(zip(cs, streams)):
            with torch.cuda.stream(s):
                got[i].append(c.call(**args[i])[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


@pytest.mark.parametrize("out", list(OUT))
@pytest.mark.parametrize("cache", [FP8, FP8_TOKEN, BF16])
def test_first_token_that_outweighs_the_others(cache, out):
    """Small weights keep their bits beside a large one: weights in f16 are off
    by 2^-25 of the largest (one term; two: 2^-35, the largest at 2^10) where
    they are subnormal, times V scales up to the largest, and the sum of the
    weights is at least the largest."""
    c = PrefixCase(20, [0] * 6 + [1] * 5, [64, 9], [5 * i + 1 for i in range(11)], q_heads=16, kv_heads=2, dim=64,
                   page=16, cache=cache)
    base = c.rng.standard_normal(64).astype(np.float32)
    c.q = synth.bf16_bits((1.5 * base + 0.3 * c.rng.standard_normal((11, 16, 64))).astype(np.float32))
    for p in (c.table[0, 0], c.table[6, 0]):
        rows = c.ref.k_pool.reshape(c.P, 2, 16, 64)[p, :, 0]
        rows[:] = synth.bf16_bits(base) if cache == BF16 else oracle.e4m3_encode(64 * base)
        if cache == FP8_TOKEN:
            c.ref.k_scale.reshape(c.P, 2, 16)[p, :, 0] = 1 / 64
            c.ref.v_scale.reshape(c.P, 2, 16)[p, :, 0] = 2.0 ** -12
    got, st = c.call(OUT[out])
    want, _, mag = c.want()
    tol = c.tolerance(want, mag, OUT[out])
    if cache != BF16:
        if cache == FP8_TOKEN:
            c.ref.v_scale[:] = c.ref.v_scale.max()
        c.tau = 0.0  # sum |v| is the mean of |v| under equal weights, times the length
        extra = c.want()[2] * c.lens[:, None, None] * 2.0 ** (-35 if out == "fp32" else -25)
        tol = tol + extra * (1 + 2.0 ** -8)
    assert not st.any() and (np.abs(got.float().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("out", list(OUT))
@pytest.mark.parametrize("cache", [FP8, FP8_TOKEN, BF16])
@pytest.mark.parametrize("most", [23.9, 35.0])
def test_largest_scores(most, cache, out):
    """Scores up to 2^23.9 (BF16 2^28.9), whose rounding is as large as the
    exponents that f16 holds, are right, of either sign; those of 2^24 and more
    (2^29) refuse their requests.  The largest score of a row leaves the others
    behind by far more than their rounding, so the output is its value: off by
    the rounding of one weight's terms and of the output.  (Half a step: a value
    between 2^e and 2^(e + 1) has steps of 2^(e - 10) in f16, so one term is off
    by 2^-11 of it, two by 2^-22; bf16 2^-8 a term, two 2^-16, three 2^-24.)"""
    c = PrefixCase(28, [0] * 6 + [1] * 5 + [-1], [40, 9], [9 * i + 1 for i in range(12)], q_heads=16, kv_heads=2,
                   dim=64, page=16, cache=cache)
    if cache == BF16 and most < 24:
        most += 5
    c.tau = 1.0
    z = scores(c)
    c.tau = float(2.0 ** most / np.abs(z[np.isfinite(z)]).max())
    for c.tau in (c.tau, -c.tau):
        got, st = c.call(OUT[out])
        if most == 35:  # every row of the groups is far beyond, in each of its pieces
            assert st.tolist() == [abi.ST_RANGE] * 11 + [0] and not got[:11].any()
        want, _, mag = c.want()
        z = np.sort(scores(c), axis=-1)
        largest = np.abs(np.where(np.isfinite(z), z, 0.0)).max(-1)
        assert (z[..., -1] - z[..., -2] > 64 + 2.0 ** -16 * largest).all()
        drop = {(True, "fp32"): -22, (True, "bf16"): -11, (False, "fp32"): -24, (False, "bf16"): -16}[cache != BF16, out]
        tol = mag * (2.0 ** drop + 2.0 ** -20)
        tol += 2.0 ** -8 * (mag + tol) if out == "bf16" else 0.0
        err = np.abs(got.float().cpu().numpy() - want)
        fine = st.cpu().numpy() == 0
        assert fine.all() or most == 35
        assert (err <= tol)[fine].all(), (np.isnan(err).sum(), np.nanmax((err / tol)[fine]))


@pytest.mark.parametrize("out", list(OUT))
@pytest.mark.parametrize("cache", [FP8, FP8_TOKEN, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_query_that_is_not_finite(bad, cache, out):
    """One element of one head's query: that row is NaN, as in the plain decode,
    the other rows of its product, its request and its group keep their bits."""
    c = PrefixCase(29, [0] * 6 + [1] * 5 + [-1], [40, 9], [9 * i + 1 for i in range(12)], q_heads=16, kv_heads=2,
                   dim=64, page=16, cache=cache)
    want = c.call(OUT[out])[0].clone()
    a = c.args()
    a["q"][2, 5, 33] = bad
    got, st = c.call(OUT[out], **a)
    rows = torch.ones(12, 16, dtype=torch.bool, device="cuda")
    rows[2, 5] = False
    assert not st.any() and torch.equal(got[rows], want[rows])
    assert got[2, 5].isnan().all()
    plain, _ = abi.paged_decode_attention(c.gpu, a["q"], a["seq_lens"], a["block_table"], None, c.tau)
    assert plain[2, 5].isnan().all()


def scores(c):
    """tau log2(e) q . k of every request and head in 64 bits; -inf past a request's length."""
    k, q = c.values("k"), synth.bf16_to_f32(c.q).astype(np.float64)
    z = np.full((c.B, c.Hq, int(c.lens.max())), -np.inf)
    for b in range(c.B):
        n = int(c.lens[b])
        kb = k[c.table[b, : -(-n // c.S)]].transpose(1, 0, 2, 3).reshape(c.H, -1, c.D)[:, :n]
        z[b, :, :n] = c.tau * math.log2(math.e) * np.einsum("hgd,htd->hgt", q[b].reshape(c.H, -1, c.D), kb).reshape(c.Hq, n)
    return z


def weight_floor(c, bits, own_max):
    """What f16 weights may be off by where they are subnormal: 2^-bits of the
    largest each, times the token's values, whose scale counts as 2^-18 of the
    prefix's largest at least; own tokens 2^-36 of their largest scale.  Without the prompt's
    scores (tau 0) the oracle's magnitude is the mean of |v|."""
    tau, scale = c.tau, c.ref.v_scale.copy()
    c.tau = 0.0
    c.ref.v_scale[:] = np.maximum(scale, scale.max() * 2.0 ** -18)
    floor = c.want()[2] * c.lens[:, None, None] * 2.0 ** -bits
    own = c.lens - np.where(c.group >= 0, c.pages[c.group], 0) * c.S
    c.tau, c.ref.v_scale[:] = tau, scale
    return floor + own[:, None, None] * 448 * own_max * 2.0 ** -36


@pytest.mark.parametrize("out", list(OUT))
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("power", [40, 14, -14, -60])
def test_values_of_any_magnitude(power, dim, out):
    """Per-token V scales up to 2^(power - 3): weights times scales stay inside
    f16's range, in the prefix and in own pages."""
    c = PrefixCase(25, [0] * 6 + [1] * 5 + [-1], [20, 9], [9 * i + 1 for i in range(12)], q_heads=16, kv_heads=2,
                   dim=dim, page=16, cache=FP8_TOKEN)
    c.ref.v_scale[:] = np.ldexp(c.ref.v_scale, power)
    got, st = c.call(OUT[out])
    want, _, mag = c.want()
    tol = c.tolerance(want, mag, OUT[out]) + weight_floor(c, 35 if out == "fp32" else 25, c.ref.v_scale.max()) * (1 + 2.0 ** -8)
    err = np.abs(got.float().cpu().numpy() - want)
    assert not st.any() and (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("out", list(OUT))
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("odd", ["zeros", "one large"])
@pytest.mark.parametrize("heavy", [False, True])
def test_v_scales_far_apart(heavy, odd, dim, out):
    """Per-token V scales of 2^-23 .. 2^-17 in a prefix, and beside them rows of
    zeros, whose scale is 1, or early rows 2^12 times as large under small
    weights: the others' weights keep their bits.  heavy: the first token
    outweighs the others."""
    c = PrefixCase(26, [0] * 6 + [1] * 5, [64, 19], [5 * i + 1 for i in range(11)], q_heads=16, kv_heads=2, dim=dim,
                   page=16, cache=FP8_TOKEN)
    ks, vs = c.ref.k_scale.reshape(c.P, 2, 16), c.ref.v_scale.reshape(c.P, 2, 16)
    k, v = c.ref.k_pool.reshape(c.P, 2, 16, dim), c.ref.v_pool.reshape(c.P, 2, 16, dim)
    vs *= np.float32(2.0 ** -14)
    own_max = vs.max()
    base = c.rng.standard_normal(dim).astype(np.float32)
    c.q = synth.bf16_bits((1.5 * base + 0.3 * c.rng.standard_normal((11, 16, dim))).astype(np.float32))
    for p in (c.table[0], c.table[6]):
        if heavy:
            k[p[0], :, 0], ks[p[0], :, 0] = oracle.e4m3_encode(64 * base), 1 / 64
        for page, slot in ((p[0], 3), (p[8], 0), (p[13], 9), (p[18], 15)):
            if odd == "zeros":
                v[page, :, slot], vs[page, :, slot] = 0, 1.0
            else:
                k[page, :, slot], ks[page, :, slot] = oracle.e4m3_encode(-64 * base), 1 / 64
                vs[page, :, slot] = own_max * 2.0 ** 12
    got, st = c.call(OUT[out])
    want, _, mag = c.want()
    tol = c.tolerance(want, mag, OUT[out]) + weight_floor(c, 35 if out == "fp32" else 25, own_max) * (1 + 2.0 ** -8)
    err = np.abs(got.float().cpu().numpy() - want)
    assert not st.any() and (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("cache", [FP8, FP8_TOKEN, BF16])
@pytest.mark.parametrize("tau", [0.0, -0.2])
def test_scales_that_are_not_positive(cache, tau):
    """Zero: every token weighs the same.  Negative: the smallest product is the largest score."""
    c = PrefixCase(18, [0, 0, -1, 0], [12], [1, 9, 21, 15], q_heads=8, kv_heads=2, dim=64, page=16, cache=cache)
    c.tau = tau
    c.assert_matches()


@pytest.mark.parametrize("cache", [FP8, BF16])
@pytest.mark.parametrize("pages", [40, 3])
def test_withheld_tile_times_out_and_context_stays_usable(cache, pages):
    """The test hook makes a CTA's first tile never arrive: the bounded waits
    give up, every request says so, and the next call is right."""
    c = PrefixCase(19, [0] * 9 + [-1], [pages], [30] * 10, q_heads=32, kv_heads=2, dim=128, page=16, cache=cache)
    _, st = c.call(flags=abi.FLAG_TEST_WITHHOLD)
    assert (st & abi.ST_TIMEOUT).all(), st
    c.assert_matches()


def test_stream_argument():
    """What a call allocates for another stream belongs to that stream."""
    c = PrefixCase(22, [0] * 12, [200], [5 * j + 1 for j in range(12)], q_heads=16, kv_heads=4, dim=128, page=16)
    want = c.call()[0].clone()
    args, side = c.args(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        got.append(c.call(**args, stream=side)[0])
        torch.empty(1 << 22, device="cuda").fill_(float("nan"))  # on the current stream, beside it
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)


@pytest.mark.parametrize("cache", [FP8, FP8_TOKEN, BF16])
def test_pages_past_four_gigabytes(cache):
    """The same batch in a small pool and at the end of one whose byte offsets
    (and, in elements, BF16 ones) pass 32 bits: the same bits."""
    c = PrefixCase(32, [0] * 9 + [1] * 3 + [-1], [10, 3], [30 * i + 1 for i in range(13)], q_heads=32, kv_heads=8,
                   dim=128, page=64, cache=cache)
    c.device()
    want, st = c.call(flags=abi.FLAG_TAG_CHECK)
    out, _, mag = c.want()
    small, far = c.gpu, 70000
    big = abi.PagedCache(far, 64, 8, 128, dtype=small.dtype, scale_mode=small.scale_mode)
    big.page_tags[-c.P:] = small.page_tags
    for name in ("k_pool", "v_pool", "k_scale", "v_scale"):
        x, y = getattr(small, name), getattr(big, name)
        if x is not None:
            y[-x.numel():] = x
    c.gpu = big
    c.table = np.where(c.table >= 0, c.table + far - c.P, -1).astype(np.int32)
    got, st2 = c.call(flags=abi.FLAG_TAG_CHECK)
    assert not st.any() and not st2.any() and torch.equal(got, want)
    # the first request's pages copied to the pool's start and read there
    n = -(-int(c.lens[0]) // 64)
    assert not abi.page_copy(big, dev_i32(c.table[0, :n]), dev_i32(np.arange(n))).any()
    c.table[0, :n], c.group[0] = np.arange(n), -1
    got, st2 = c.call()
    assert not st2.any()
    c.assert_close(got, out, mag, torch.float32)


@pytest.mark.parametrize("batch,n_groups,Hq,H", [(65535, 4096, 1, 1), (4096, 4096, 12, 2), (300, 1, 512, 1)])
def test_largest_batches_groups_and_head_groups(batch, n_groups, Hq, H):
    """Against the plain decode of the same tables: fp32 sums of products of
    either, each within the tolerance of the other tests (here, as bounds of
    all rows: scores of at most 2^6, contexts of at most 100 tokens)."""
    g = torch.Generator(device="cuda").manual_seed(6)
    D, S = 64, 16
    pages = torch.randint(0, 3, (n_groups,), generator=g, device="cuda", dtype=torch.int32)
    group = torch.randint(-1, n_groups, (batch,), generator=g, device="cuda", dtype=torch.int32)
    skip = torch.where(group < 0, 0, pages[group.clamp(min=0).long()])
    lens = (skip * S + torch.randint(1, 3 * S + 1, (batch,), generator=g, device="cuda")).int()
    P = 2 * n_groups + 3 * batch
    own = (2 * n_groups + torch.arange(3 * batch, device="cuda", dtype=torch.int32)).view(batch, 3)
    cols = torch.arange(5, device="cuda")[None]
    table = torch.where(cols < skip[:, None], 2 * group.clamp(min=0)[:, None] + cols,
                        own.gather(1, (cols - skip[:, None]).clamp(0, 2).long())).int()
    cache = abi.PagedCache(P, S, H, D)
    for pool in (cache.k_pool, cache.v_pool):  # codes of magnitudes below 2, of either sign
        pool.copy_(torch.randint(0, 64, pool.shape, generator=g, device="cuda", dtype=torch.uint8))
        pool += 128 * torch.randint(0, 2, pool.shape, generator=g, device="cuda", dtype=torch.uint8)
    q = torch.randn((batch, Hq, D), generator=g, device="cuda").bfloat16()
    got, st = abi.paged_decode_attention_prefix(cache, q, lens, table, None, group, pages, 0.125, max_splits=2)
    want, st2 = abi.paged_decode_attention(cache, q, lens, table, None, 0.125, max_splits=2)
    assert not st.any() and not st2.any()
    # |v| < 2; scores off by (64 + 4) 2^-24 x 2^6, twice, weights by 2^-21, sums by 100 x 2^-24, in both calls
    assert ((got - want).abs() <= 2 * 2 * (2 * 68 * 64 * 2.0 ** -24 * math.log(2) + 2.0 ** -20 + 200 * 2.0 ** -24)).all()


def test_a_refused_call_enqueues_nothing():
    """More KV heads than the split kernel takes: workspace, output and status
    stay as they were."""
    H, B = 4097, 2
    cache = abi.PagedCache(2, 16, H, 64, fill=0)
    ws = torch.full((1 << 29,), 0xEE, dtype=torch.uint8, device="cuda")  # enough for these sizes
    out = torch.full((B, H, 64), 7.0, device="cuda")
    st = torch.full((B,), -5, dtype=torch.int32, device="cuda")
    q = torch.zeros((B, H, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(abi.PfkvError):
        abi.paged_decode_attention_prefix(cache, q, dev_i32(np.array([20, 20])), dev_i32(np.array([[0, 1], [0, 1]])), None,
                                          dev_i32(np.array([0, 0])), dev_i32(np.array([1])), 0.1, max_splits=2,
                                          workspace=ws, out=out, status=st)
    torch.cuda.synchronize()
    assert (ws == 0xEE).all() and (out == 7.0).all() and (st == -5).all()


def test_fork_decode_release_together():
    """One prompt forked into samples that decode a few steps each, reading the
    prompt's pages once, and are given back: outputs against the oracle, and
    the pool as it was."""
    S, H, Hq, D, P, B, MP, n0 = 16, 2, 8, 64, 80, 7, 10, 100
    rng = np.random.default_rng(30)
    cache = abi.PagedCache(P, S, H, D)
    cache.k_scale.fill_(0.01)
    cache.v_scale.fill_(0.01)
    alloc = abi.PageAllocator(P)
    table = torch.full((B, MP), -1, dtype=torch.int32, device="cuda")
    tags = torch.zeros((B, MP), dtype=torch.int32, device="cuda")
    pages, ptags, _ = alloc.alloc(-(-n0 // S), cache.page_tags)
    table[0, : pages.numel()], tags[0, : pages.numel()] = pages, ptags

    def rows(n):
        return synth.bf16_bits(rng.standard_normal((n, H, D), dtype=np.float32))

    prompt = rows(n0), rows(n0)
    st = abi.kv_append_quantize(cache, dev_bf16(prompt[0]), dev_bf16(prompt[1]), dev_i32(np.arange(n0)), table, tags,
                                flags=abi.FLAG_TAG_CHECK, row_req=dev_i32(np.zeros(n0, np.int32)), batch=B)
    assert not st.any()
    kids = list(range(1, B))
    st = alloc.fork(cache, dev_i32(np.zeros(B - 1, np.int32)), dev_i32(np.array(kids)),
                    dev_i32(np.full(B - 1, n0, np.int32)), table, tags, flags=abi.FLAG_TAG_CHECK)
    assert not st.any()
    group, shared = torch.zeros(B, dtype=torch.int32, device="cuda"), dev_i32(np.array([n0 // S]))
    c = PrefixCase(31, [0] * B, [n0 // S], [n0 % S] * B, q_heads=Hq, kv_heads=H, dim=D, page=S)
    c.P, c.gpu = P, cache
    for step in range(20):
        lens = np.full(B, n0 + step + 1, np.int32)
        if lens[0] % S == 1:  # a fresh page for each
            pages, ptags, s1 = alloc.alloc(B, cache.page_tags)
            assert not s1.any()
            table[:, (lens[0] - 1) // S], tags[:, (lens[0] - 1) // S] = pages, ptags
        q = synth.bf16_bits(rng.standard_normal((B, Hq, D), dtype=np.float32))
        out, st = abi.paged_decode_attention_prefix(cache, dev_bf16(q), dev_i32(lens), table, tags, group, shared,
                                                    0.125, flags=abi.FLAG_TAG_CHECK, k_new=dev_bf16(rows(B)),
                                                    v_new=dev_bf16(rows(B)))
        assert not st.any()
        if step in (0, 11, 12, 19):
            c.table, c.tags = table.cpu().numpy(), tags.cpu().numpy().view(np.uint32)
            c.lens, c.q, c.tau = lens, q, 0.125
            c.ref = oracle.Cache(P, S, H, D, page_tags=cache.page_tags.cpu().numpy().view(np.uint32),
                                 k_scale=cache.k_scale.cpu().numpy(), v_scale=cache.v_scale.cpu().numpy())
            c.ref.k_pool[:], c.ref.v_pool[:] = cache.k_pool.cpu().numpy(), cache.v_pool.cpu().numpy()
            # the codec's NaN codes do not occur in written slots; unwritten ones are not read by the oracle
            c.ref.k_pool[(c.ref.k_pool & 0x7F) == 0x7F] = 0
            c.ref.v_pool[(c.ref.v_pool & 0x7F) == 0x7F] = 0
            want, st_ref, mag = c.want(abi.FLAG_TAG_CHECK)
            assert not st_ref.any()
            c.assert_close(out, want, mag, torch.float32, step)
    used = -(-(n0 + 20) // S)
    assert not alloc.release(table[1:, :used].reshape(-1).contiguous()).any()
    assert alloc.free_count() == P - used and not alloc.refs.any()
    src, dst, n = alloc.compact(cache, table[:1].contiguous(), tags[:1].contiguous())
    assert not alloc.release(table[0, :used].contiguous() if int(n.item()) == 0 else
                             torch.arange(used, dtype=torch.int32, device="cuda")).any()
    assert alloc.free_count() == P


def test_wrong_arguments_are_refused():
    c = PrefixCase(40, [0, 0], [2], [3, 4], q_heads=4, kv_heads=2, dim=64, page=16)
    c.device()
    with pytest.raises(ValueError):
        c.call(prefix_group=dev_i32(np.array([0])))
    with pytest.raises(ValueError):
        c.call(out=torch.empty(2, 4, 64, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        c.call(q=dev_bf16(c.q).transpose(0, 1))
    with pytest.raises(ValueError):
        c.call(q=torch.zeros(2, 4, 32, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(abi.PfkvError):
        c.call(workspace=torch.empty(512, dtype=torch.uint8, device="cuda"))
    with pytest.raises(abi.PfkvError):
        c.call(k_new=torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda"))
    for tau in (float("nan"), float("inf")):
        with pytest.raises(abi.PfkvError):
            c.tau = tau
            c.call()
    c.tau = 0.1
    with pytest.raises(abi.PfkvError):
        c.call(block_tags=None, flags=abi.FLAG_TAG_CHECK)
