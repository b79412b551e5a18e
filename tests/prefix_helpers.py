"""Batches whose groups share prefixes, on the GPU and in the oracle, and how
far an output may be from the oracle's."""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle
from gpu_helpers import dev_bf16, dev_i32
from paged_fp8_kv_quantize_gb300 import abi, synth

FP8, FP8_TOKEN, BF16 = "fp8", "fp8_token", "bf16"


class PrefixCase:
    """group: the group of each request (-1: none); pages: shared pages of each
    group; own: tokens past the prefix of each request."""

    def __init__(self, seed, group, pages, own, *, q_heads, kv_heads, dim, page, cache=FP8, spread=1.0, room=0):
        rng = np.random.default_rng(seed)
        self.rng, self.S, self.D, self.H, self.Hq, self.cache_kind = rng, page, dim, kv_heads, q_heads, cache
        B = len(group)
        self.group, self.pages = np.array(group, np.int32), np.array(pages, np.int32)
        pre = np.array([pages[g] if g >= 0 else 0 for g in group], np.int64)
        self.lens = (pre * page + np.array(own)).astype(np.int32)
        need = -(-(self.lens + room) // page)
        MP = int(need.max()) + 1
        P = int(sum(pages) + (need - pre).sum()) + 5
        self.P, self.B, self.MP = P, B, MP
        perm = rng.permutation(P).tolist()
        shared = [[perm.pop() for _ in range(n)] for n in pages]
        self.table = np.full((B, MP), -1, np.int32)
        for b in range(B):
            row = list(shared[group[b]]) if group[b] >= 0 else []
            row += [perm.pop() for _ in range(int(need[b]) - len(row))]
            self.table[b, : len(row)] = row
        self.page_tags = rng.integers(0, 1 << 32, size=P, dtype=np.uint64).astype(np.uint32)
        self.tags = np.where(self.table >= 0, self.page_tags[np.maximum(self.table, 0)], 0).astype(np.uint32)
        self.tau = spread / math.sqrt(dim)
        self.q = synth.bf16_bits(rng.standard_normal((B, q_heads, dim), dtype=np.float32))
        dtype = oracle.DTYPE_BF16 if cache == BF16 else oracle.DTYPE_FP8
        mode = oracle.SCALE_PER_TOKEN if cache == FP8_TOKEN else oracle.SCALE_PER_HEAD
        self.ref = oracle.Cache(P, page, kv_heads, dim, dtype=dtype, scale_mode=mode, page_tags=self.page_tags)
        n = P * kv_heads * page
        for name in ("k", "v"):
            x = rng.standard_normal((n, dim), dtype=np.float32)
            if cache == BF16:
                getattr(self.ref, name + "_pool")[:] = synth.bf16_bits(x).reshape(-1)
                continue
            codes = oracle.e4m3_encode(x.reshape(-1) * np.float32(64.0))
            getattr(self.ref, name + "_pool")[:] = codes
            s = getattr(self.ref, name + "_scale")
            s[:] = (2.0 ** rng.uniform(-9, -3, size=s.size) if cache == FP8_TOKEN else
                    rng.uniform(0.5, 2.0, size=s.size) / 64).astype(np.float32)

    def device(self):
        r = self.ref
        bf = self.cache_kind == BF16
        c = abi.PagedCache(self.P, self.S, self.H, self.D,
                           dtype=abi.DTYPE_BF16 if bf else abi.DTYPE_FP8_E4M3, scale_mode=r.scale_mode)
        for name in ("k", "v"):
            pool = torch.from_numpy(getattr(r, name + "_pool").view(np.int16 if bf else np.uint8))
            getattr(c, name + "_pool").copy_(pool.view(torch.bfloat16) if bf else pool)
            if not bf:
                getattr(c, name + "_scale").copy_(torch.from_numpy(getattr(r, name + "_scale")))
        c.page_tags.copy_(dev_i32(self.page_tags))
        self.gpu = c
        return c

    def args(self):
        return dict(q=dev_bf16(self.q), seq_lens=dev_i32(self.lens), block_table=dev_i32(self.table),
                    block_tags=dev_i32(self.tags), prefix_group=dev_i32(self.group),
                    prefix_pages=dev_i32(self.pages))

    def call(self, out_dtype=torch.float32, flags=0, max_splits=64, **kw):
        if not hasattr(self, "gpu"):
            self.device()
        args = kw if "q" in kw and "prefix_pages" in kw else {**self.args(), **kw}
        return abi.paged_decode_attention_prefix(self.gpu, softmax_scale=self.tau, flags=flags, max_splits=max_splits,
                                                 out_dtype=out_dtype, **args)

    def want(self, flags=0):
        """The oracle's output and status, and sum p |v| / l of every value."""
        out, st = self.ref.decode(self.q, self.lens, self.table, self.tags, self.tau, flags=flags, threads=8)
        v = self.ref.v_pool.copy()
        self.ref.v_pool &= np.array(0x7FFF if self.cache_kind == BF16 else 0x7F, v.dtype)
        mag, _ = self.ref.decode(self.q, self.lens, self.table, self.tags, self.tau, flags=flags, threads=8)
        self.ref.v_pool[:] = v
        return out, st, mag

    def tolerance(self, out, mag, out_dtype):
        """A score z = tau log2(e) q.k is a sum of D exact products in fp32, off
        by at most (D + 4) 2^-24 |tau| log2(e) sum |q k|; a weight 2^(z - m) then by the
        factor e^(2 dz ln 2), 2^-21 from the exponential and its scales, and
        what its 16-bit terms drop (FP8: 2^-22 or, for a bf16 output, 2^-11;
        BF16: 2^-24 or 2^-16); sums of L weights by L 2^-24, in numerator and
        denominator.  All of it scales sum p |v| / l.  Then the output's own
        rounding, half a step."""
        q = np.abs(synth.bf16_to_f32(self.q).astype(np.float64))
        kmax = np.abs(self.values("k")).max(axis=(0, 2))  # [H][D]
        z = np.einsum("bhd,hd->bh", q, np.repeat(kmax, self.Hq // self.H, axis=0)) * abs(self.tau) * math.log2(math.e)
        dz = (self.D + 4) * 2.0 ** -24 * z
        fp32 = out_dtype == torch.float32
        drop = (2.0 ** -24 if fp32 else 2.0 ** -16) if self.cache_kind == BF16 else (2.0 ** -22 if fp32 else 2.0 ** -11)
        eps = 2 * (2 * dz * math.log(2) + 2.0 ** -21 + self.lens[:, None].astype(np.float64).clip(min=0) * 2.0 ** -24)
        tol = mag * (eps[..., None] + drop) + 2.0 ** -24 * np.abs(out)
        return tol if fp32 else tol + 2.0 ** -8 * (np.abs(out) + tol)

    def values(self, which):
        pool = getattr(self.ref, which + "_pool")
        x = synth.bf16_to_f32(pool) if self.cache_kind == BF16 else oracle.e4m3_decode(pool)
        x = x.astype(np.float64).reshape(self.P, self.H, self.S, self.D)
        if self.cache_kind == BF16:
            return x
        s = getattr(self.ref, which + "_scale").astype(np.float64)
        return x * (s.reshape(self.P, self.H, self.S, 1) if self.cache_kind == FP8_TOKEN else s[None, :, None, None])

    def assert_matches(self, out_dtype=torch.float32, flags=0, where="", **kw):
        got, st = self.call(out_dtype, flags, **kw)
        torch.cuda.synchronize()
        out, st_ref, mag = self.want(flags)
        assert np.array_equal(st.cpu().numpy().view(np.uint32), st_ref), (where, st, st_ref)
        self.assert_close(got, out, mag, out_dtype, where)
        return got

    def assert_close(self, got, out, mag, out_dtype, where=""):
        err = np.abs(got.float().cpu().numpy().astype(np.float64) - out)
        tol = self.tolerance(out, mag, out_dtype)
        bad = ~(err <= tol)
        assert not bad.any(), (where, np.argwhere(bad)[:5], err[bad][:5], tol[bad][:5])
