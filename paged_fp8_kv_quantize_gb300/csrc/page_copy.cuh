// page_copy.cuh -- one block copies a slab of one page of a cache to another
// page of the same cache: codes (or bf16 values) of K and V, and the
// per-token scales.  Used by the page copy, by the fork (the partly filled
// last page) and by the compaction.
//
// A page's K rows of all heads are one contiguous range of its pool, V's
// likewise, so a whole page is two contiguous copies; the first `slots` rows
// of every head are num_kv_heads runs of slots rows per pool.  The bytes of a
// page are numbered K first, then V, in vectors of kVec bytes, and a slab is
// kSlabVecs of them: 16 KB, so that a page of the usual shapes gives one to
// a few blocks, each with four independent loads per thread in flight.
#pragma once

#include "pfkv_internal.h"

namespace pfkv {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kSlabVecs = kCopyThreads * kCopyUnroll;

// Copies are 16 bytes wide where rows are (every offset inside a pool is a
// multiple of the row); the other rows are multiples of 8 bytes.
__host__ __device__ inline int copy_vec_bytes(const pfkv_cache &c) {
  const int e = c.dtype == PFKV_DTYPE_FP8_E4M3 ? 1 : 2;
  return (c.head_dim * e) % 16 == 0 && (c.v_head_dim * e) % 16 == 0 ? 16 : 8;
}

// Slabs of a whole page.
inline long long copy_slabs(const pfkv_cache &c) {
  const long long e = c.dtype == PFKV_DTYPE_FP8_E4M3 ? 1 : 2;
  const long long row = (long long)(c.head_dim + (c.kv_shared ? 0 : c.v_head_dim)) * e;
  const long long vecs = row * c.num_kv_heads * c.page_size / copy_vec_bytes(c);
  return (vecs + kSlabVecs - 1) / kSlabVecs;
}

// The whole block (kCopyThreads threads): slab `slab` of the first `slots`
// slots (1 .. page_size) of page src into page dst.  Slab 0 also takes the
// per-token scales.
template <typename V>
__device__ __forceinline__ void copy_page_slab(const pfkv_cache &c, int src, int dst, int slots, long long slab) {
  constexpr int kVec = sizeof(V);
  const int e = c.dtype == PFKV_DTYPE_FP8_E4M3 ? 1 : 2;
  const int H = c.num_kv_heads, S = c.page_size, t = threadIdx.x;
  // vectors of one head: a full page's run and the run that is copied
  const long long hk = (long long)S * c.head_dim * e / kVec, hv = c.kv_shared ? 0 : (long long)S * c.v_head_dim * e / kVec;
  const long long nk = (long long)slots * c.head_dim * e / kVec, nv = c.kv_shared ? 0 : (long long)slots * c.v_head_dim * e / kVec;
  const long long k_total = nk * H, total = k_total + nv * H;
  const long long first = slab * kSlabVecs + t;
  const V *k_src = reinterpret_cast<const V *>(c.k_pool) + (long long)src * H * hk;
  V *k_dst = reinterpret_cast<V *>(c.k_pool) + (long long)dst * H * hk;
  const V *v_src = reinterpret_cast<const V *>(c.v_pool) + (long long)src * H * hv;
  V *v_dst = reinterpret_cast<V *>(c.v_pool) + (long long)dst * H * hv;
  const bool whole = slots == S;
  V x[kCopyUnroll];
  long long at[kCopyUnroll];  // vector offset inside the page, K or V
#pragma unroll
  for (int j = 0; j < kCopyUnroll; ++j) {
    const long long i = first + (long long)j * kCopyThreads;
    const bool is_v = i >= k_total;
    long long o = is_v ? i - k_total : i;
    if (!whole) {
      const unsigned run = (unsigned)(is_v ? nv : nk);  // page runs fit 32 bits: at most 2^24 rows' worth of a head
      if (o >> 32) {
        o = o / run * (is_v ? hv : hk) + o % run;
      } else if (run) {
        const unsigned h = (unsigned)o / run;
        o = (long long)h * (is_v ? hv : hk) + ((unsigned)o - h * run);
      }
    }
    at[j] = o;
    if (i < total) x[j] = (is_v ? v_src : k_src)[o];
  }
#pragma unroll
  for (int j = 0; j < kCopyUnroll; ++j) {
    const long long i = first + (long long)j * kCopyThreads;
    if (i < total) (i >= k_total ? v_dst : k_dst)[at[j]] = x[j];
  }
  if (slab == 0 && c.dtype == PFKV_DTYPE_FP8_E4M3 && c.scale_mode == PFKV_SCALE_PER_TOKEN) {
    const long long rs = (long long)src * H * S, rd = (long long)dst * H * S;
    for (long long i = t; i < (long long)H * slots; i += kCopyThreads) {
      const long long o = i / slots * S + i % slots;
      c.k_scale[rd + o] = c.k_scale[rs + o];
      if (!c.kv_shared) c.v_scale[rd + o] = c.v_scale[rs + o];
    }
  }
}

}  // namespace
}  // namespace pfkv
