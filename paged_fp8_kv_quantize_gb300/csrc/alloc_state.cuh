// alloc_state.cuh -- the page allocator's device state, shared by the kernels
// that work on it (alloc.cu: init, alloc, free, realloc; share.cu: fork,
// release; compact.cu: compact).  Everything here has internal linkage.
#pragma once

#include <climits>

#include "pfkv_internal.h"

namespace pfkv {
namespace {

constexpr int kAT = 1024;  // threads of the single-CTA kernels; also init's chunk

struct AllocHdr {
  int num_pages;
  int free_count;
  int ticket;  // blocks of a fork's check or a compaction's count that are done; zero between calls
  int pad[61];
};

__host__ __device__ inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

struct AllocLayout {
  size_t stack, mark, held, counts, total;
};

__host__ __device__ inline AllocLayout alloc_layout(int P) {
  AllocLayout L;
  L.stack = 256;
  L.mark = L.stack + round256(size_t(P) * 4);
  L.held = L.mark + round256(size_t(P) * 4);
  L.counts = L.held + round256(size_t(P));
  L.total = L.counts + round256((size_t((P + kAT - 1) / kAT) + 1) * 4);
  return L;
}

struct AllocView {
  AllocHdr *hdr;
  int *stack, *mark;
  uint8_t *held;
  int *counts;
};

__device__ inline AllocView view(void *state) {
  uint8_t *base = static_cast<uint8_t *>(state);
  AllocView v;
  v.hdr = reinterpret_cast<AllocHdr *>(base);
  const AllocLayout L = alloc_layout(v.hdr->num_pages);
  v.stack = reinterpret_cast<int *>(base + L.stack);
  v.mark = reinterpret_cast<int *>(base + L.mark);
  v.held = base + L.held;
  v.counts = reinterpret_cast<int *>(base + L.counts);
  return v;
}

// Exclusive scan of one flag per thread over the block (1024 threads);
// returns this thread's rank, total in *total.  Uses s_warp[32].
__device__ inline int block_rank(bool flag, int *s_warp, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned bal = __ballot_sync(0xffffffffu, flag);
  const int in_warp = __popc(bal & ((1u << lane) - 1u));
  if (lane == 0) s_warp[warp] = __popc(bal);
  __syncthreads();
  if (warp == 0) {
    const int c = s_warp[lane];
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    s_warp[lane] = incl - c;
    if (lane == 31) s_warp[32] = incl;
  }
  __syncthreads();
  const int r = s_warp[warp] + in_warp;
  *total = s_warp[32];
  __syncthreads();  // s_warp is reused by the next call
  return r;
}

}  // namespace
}  // namespace pfkv
