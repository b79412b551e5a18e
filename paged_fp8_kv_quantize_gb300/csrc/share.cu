// share.cu -- pages held by several requests: fork and release.
//
// A fork gives a child row of the block table the parent's context without
// copying it: the full pages are shared (one more holder each), and only the
// partly filled last page, which both sides go on writing, is copied into a
// fresh page, whose tag advances as on every hand-out.  A release takes one
// holder off each listed page and returns the page to the free list when
// nobody holds it any more.  page_refs[p] counts the holders of page p
// beyond the first, so a pool that has never forked is all zeros and a
// release there is a free.
//
// Both are bound by latency: their bytes (8 per shared table entry, a page
// per fork) take a microsecond or two, and the rest is dependent look-ups.
// Fork: a check with one block per fork (bounds, held, tag of every page),
// whose last block to finish hands out the new pages in list order; then a
// grid that copies table entries, counts holders and copies the last pages.
#include "alloc_state.cuh"
#include "page_copy.cuh"
#include "pfkv_device.cuh"

namespace pfkv {

namespace {

// ---------------------------------------------------------------- fork

struct ForkArgs {
  void *state;
  uint32_t *page_tags;
  int *page_refs;
  pfkv_cache c;
  const int *parents, *children, *lens;
  int n;
  int *table;
  uint32_t *tags;  // NULL: no tags are kept
  int batch, MP;
  uint32_t flags;
  uint32_t *status;  // [n]
};

// Block i checks fork i; the block that finishes last hands out the pages.
__global__ void __launch_bounds__(kAT) fork_check_kernel(const ForkArgs f) {
  __shared__ uint32_t s_bits;
  __shared__ int s_last;
  __shared__ int s_warp[33];
  const int i = blockIdx.x, t = threadIdx.x;
  AllocView v = view(f.state);
  if (t == 0) s_bits = 0u;
  __syncthreads();
  const int S = f.c.page_size, P = f.c.num_pages;
  const int par = f.parents[i], chi = f.children[i], len = f.lens[i];
  uint32_t bits = 0u;
  if (v.hdr->num_pages != P) bits |= PFKV_ST_PAGE_OOB;  // not this cache's allocator
  if (par < 0 || par >= f.batch || chi < 0 || chi >= f.batch) bits |= PFKV_ST_BAD_ROW;
  if (len < 0 || (long long)len > (long long)f.MP * S) bits |= PFKV_ST_BAD_LEN;
  // a child that an earlier entry makes, or that any entry forks from
  for (int j = t; j < f.n; j += kAT)
    if ((j < i && f.children[j] == chi) || f.parents[j] == chi) bits |= PFKV_ST_DUPLICATE;
  if (!(bits & (PFKV_ST_PAGE_OOB | PFKV_ST_BAD_ROW | PFKV_ST_BAD_LEN))) {
    const int used = (int)(((unsigned)len + (unsigned)S - 1u) / (unsigned)S);
    const int *row = f.table + (size_t)par * f.MP;
    const uint32_t *want = f.tags + (size_t)par * f.MP;  // read under the tag check only
#pragma unroll 4
    for (int k = t; k < used; k += kAT) {
      const int p = row[k];
      if (p < 0 || p >= P) {
        bits |= PFKV_ST_PAGE_OOB;
      } else {
        if (!v.held[p]) bits |= PFKV_ST_NOT_HELD;
        if ((f.flags & PFKV_FLAG_TAG_CHECK) && f.page_tags[p] != want[k]) bits |= PFKV_ST_STALE_TAG;
      }
    }
  }
  if (bits) atomicOr(&s_bits, bits);
  __syncthreads();
  if (t == 0) {
    f.status[i] = s_bits;
    __threadfence();
    s_last = atomicAdd(&v.hdr->ticket, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();

  // The last block: one fresh page for each sound fork whose length ends
  // inside a page, in list order; with too few free pages nothing is taken.
  const int fc = v.hdr->free_count;
  long long need = 0;
  for (int base = 0; base < f.n; base += kAT) {
    const int j = base + t;
    const bool takes = j < f.n && __ldcg(&f.status[j]) == 0u && f.lens[j] % S != 0;
    need += __syncthreads_count(takes);
  }
  const bool enough = need <= fc;
  int taken = 0;
  for (int base = 0; base < f.n; base += kAT) {
    const int j = base + t;
    const bool sound = j < f.n && __ldcg(&f.status[j]) == 0u;
    if (!enough) {
      if (sound) f.status[j] = PFKV_ST_NO_PAGES;
      continue;
    }
    const bool takes = sound && f.lens[j] % S != 0;
    int total;
    const int r = block_rank(takes, s_warp, &total);
    if (takes) {
      const int p = v.stack[fc - 1 - taken - r];
      v.held[p] = 1;
      const uint32_t tag = f.page_tags[p] + 1u;
      f.page_tags[p] = tag;
      const size_t at = (size_t)f.children[j] * f.MP + f.lens[j] / S;
      f.table[at] = p;
      if (f.tags) f.tags[at] = tag;
    }
    taken += total;
  }
  if (t == 0) {
    v.hdr->free_count = fc - taken;
    v.hdr->ticket = 0;
  }
}

constexpr int kForkEntries = 4 * kCopyThreads;  // table entries per block

// blockIdx.x = fork; blockIdx.y walks its units: slabs of the last page,
// then ranges of table entries.
template <typename V>
__global__ void __launch_bounds__(kCopyThreads) fork_apply_kernel(const ForkArgs f, long long n_slabs,
                                                                  long long n_units) {
  pdl_wait();
  const int i = blockIdx.x, t = threadIdx.x;
  if (f.status[i]) return;
  const int S = f.c.page_size, len = f.lens[i];
  const int full = len / S, tail = len - full * S;
  const size_t from = (size_t)f.parents[i] * f.MP, to = (size_t)f.children[i] * f.MP;
  for (long long u = blockIdx.y; u < n_units; u += gridDim.y) {
    if (u < n_slabs) {
      if (tail) copy_page_slab<V>(f.c, f.table[from + full], f.table[to + full], tail, u);
      continue;
    }
    const long long k0 = (u - n_slabs) * kForkEntries;
    if (k0 >= full) break;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long k = k0 + j * kCopyThreads + t;
      if (k < full) {
        const int p = f.table[from + k];
        f.table[to + k] = p;
        if (f.tags) f.tags[to + k] = f.tags[from + k];
        atomicAdd(&f.page_refs[p], 1);
      }
    }
  }
}

// ---------------------------------------------------------------- release
//
// The list is processed as if in order: a page with h holders may be listed
// h times, and the h-th time returns it to the free list (at that place of the
// list).  One listed more often, a caller's mistake, goes back where it is
// listed first, and its other listings are NOT_HELD.  Three passes:
//   count: how often each held page is listed (c), in its scratch word, as
//          INT_MAX - c.
//   sort:  a page with c < h stays held (kShared).  One with c = h is
//          returned where it is listed last (kLast): the entries' largest
//          index is found with atomicMin of -(index + 1) on the same word;
//          c > h (kOver) where it is listed first: atomicMin of
//          index - (2^31 - 1), which lies below all of those.
//   apply: kShared entries take one holder off; the others are walked by one
//          block in list order, which pushes the returned pages.
// Classes stand in page_status between the passes.  Lists of up to
// kReleaseOneBlock entries run all three in one block (one launch).
enum { kShared = 0x10000u, kLast = 0x20000u, kOver = 0x40000u };
constexpr int kOverBase = -INT_MAX;      // its entry i is marked kOverBase + i, below -(i + 1) as n < 2^30
constexpr int kReleaseOneBlock = 4096;
// Consecutive entries per thread of the ordered walk (64 rows of 1875 shared
// pages given back: the apply kernel took 42 us with 4, 16 with 16).
constexpr int kReleasePer = 16;

struct ReleaseArgs {
  void *state;
  int *page_refs;
  const int *pages;
  int n;
  uint32_t *status;
};

__device__ __forceinline__ int holders(const ReleaseArgs &r, int p) { return max(__ldcg(&r.page_refs[p]), 0) + 1; }

__device__ __forceinline__ void release_count(const ReleaseArgs &r, const AllocView &v, int P, int i) {
  const int p = r.pages[i];
  if (p < 0 || p >= P)
    r.status[i] = PFKV_ST_PAGE_OOB;
  else if (!v.held[p])
    r.status[i] = PFKV_ST_NOT_HELD;
  else {
    r.status[i] = kShared;
    atomicSub(&v.mark[p], 1);
  }
}

__device__ __forceinline__ void release_sort(const ReleaseArgs &r, const AllocView &v, int i) {
  if (__ldcg(&r.status[i]) != kShared) return;
  const int p = r.pages[i];
  const int m = __ldcg(&v.mark[p]);
  bool over;
  if (m < 0) {  // another entry has marked the page
    over = m < kOverBase / 2;
  } else {
    const int c = INT_MAX - m, h = holders(r, p);
    if (c < h) return;
    over = c > h;
  }
  r.status[i] = over ? kOver : kLast;
  atomicMin(&v.mark[p], over ? kOverBase + i : -(i + 1));
}

__device__ __forceinline__ void release_shared(const ReleaseArgs &r, const AllocView &v, int i) {
  if (__ldcg(&r.status[i]) != kShared) return;
  const int p = r.pages[i];
  atomicSub(&r.page_refs[p], 1);
  v.mark[p] = INT_MAX;
  r.status[i] = 0u;
}

// One block, in list order: pushes the pages that nobody holds any more.
__device__ __forceinline__ void release_push(const ReleaseArgs &r, const AllocView &v, int *s_warp) {
  const int fc = v.hdr->free_count, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const bool vec = (reinterpret_cast<uintptr_t>(r.status) & 15u) == 0;
  int pushed = 0;
  for (int base = 0; base < r.n; base += kAT * kReleasePer) {
    const long long i0 = (long long)base + t * kReleasePer;
    uint32_t st[kReleasePer];
    if (vec && i0 + kReleasePer <= r.n) {
#pragma unroll
      for (int j = 0; j < kReleasePer; j += 4) {
        const uint4 x = __ldcg(reinterpret_cast<const uint4 *>(r.status + i0 + j));
        st[j] = x.x; st[j + 1] = x.y; st[j + 2] = x.z; st[j + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kReleasePer; ++j) st[j] = i0 + j < r.n ? __ldcg(&r.status[i0 + j]) : 0u;
    }
    uint32_t push = 0u;  // bit j: entry j returns its page
#pragma unroll
    for (int j = 0; j < kReleasePer; ++j) {
      if (!(st[j] & (kLast | kOver))) continue;
      const int i = (int)i0 + j, p = r.pages[i];
      const bool over = st[j] == kOver, back = __ldcg(&v.mark[p]) == (over ? kOverBase + i : -(i + 1));
      push |= (uint32_t)back << j;
      r.status[i] = over && !back ? PFKV_ST_NOT_HELD : 0u;
    }
    const int cnt = __popc(push);
    // exclusive scan of cnt over the block
    int incl = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      const int wsum = s_warp[lane];
      int wincl = wsum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, wincl, o);
        if (lane >= o) wincl += y;
      }
      s_warp[lane] = wincl - wsum;
      if (lane == 31) s_warp[32] = wincl;
    }
    __syncthreads();
    int at = fc + pushed + s_warp[warp] + incl - cnt;
    for (uint32_t m = push; m; m &= m - 1) v.stack[at++] = r.pages[i0 + __ffs(m) - 1];
    pushed += s_warp[32];
    __syncthreads();  // s_warp is reused, and the pushed ids are read below
  }
  for (int k = t; k < pushed; k += kAT) {
    const int p = __ldcg(&v.stack[fc + k]);
    v.held[p] = 0;
    v.mark[p] = INT_MAX;
    r.page_refs[p] = 0;
  }
  if (t == 0) v.hdr->free_count = fc + pushed;
}

__global__ void __launch_bounds__(kAT) release_one_block_kernel(const ReleaseArgs r) {
  __shared__ int s_warp[33];
  AllocView v = view(r.state);
  const int P = v.hdr->num_pages;
  for (int i = threadIdx.x; i < r.n; i += kAT) release_count(r, v, P, i);
  __syncthreads();
  for (int i = threadIdx.x; i < r.n; i += kAT) release_sort(r, v, i);
  __syncthreads();
  for (int i = threadIdx.x; i < r.n; i += kAT) release_shared(r, v, i);
  release_push(r, v, s_warp);
}

__global__ void __launch_bounds__(256) release_count_kernel(const ReleaseArgs r) {
  AllocView v = view(r.state);
  const int P = v.hdr->num_pages;
  const long long i = blockIdx.x * 256LL + threadIdx.x;
  if (i < r.n) release_count(r, v, P, (int)i);
}

__global__ void __launch_bounds__(256) release_sort_kernel(const ReleaseArgs r) {
  pdl_wait();
  AllocView v = view(r.state);
  const long long i = blockIdx.x * 256LL + threadIdx.x;
  if (i < r.n) release_sort(r, v, (int)i);
}

// Block 0 walks the list; the others take holders off shared pages.
__global__ void __launch_bounds__(kAT) release_apply_kernel(const ReleaseArgs r) {
  __shared__ int s_warp[33];
  pdl_wait();
  AllocView v = view(r.state);
  if (blockIdx.x == 0) {
    release_push(r, v, s_warp);
    return;
  }
  const long long i = (blockIdx.x - 1) * (long long)kAT + threadIdx.x;
  if (i < r.n) release_shared(r, v, (int)i);
}

}  // namespace

int launch_page_fork(void *state, uint32_t *page_tags, int *page_refs, const pfkv_cache &c, const int *parents,
                     const int *children, const int *lens, int n, int *block_table, uint32_t *block_tags, int batch,
                     int max_pages, uint32_t flags, uint32_t *status, cudaStream_t s) {
  const ForkArgs f{state,       page_tags,  page_refs, c,         parents, children, lens, n,
                   block_table, block_tags, batch,     max_pages, flags,   status};
  fork_check_kernel<<<n, kAT, 0, s>>>(f);
  int rc = cuda_ok(cudaGetLastError(), "fork check launch");
  if (rc) return rc;
  const long long slabs = copy_slabs(c);
  const long long units = slabs + (max_pages + kForkEntries - 1) / kForkEntries;
  const dim3 grid(n, (unsigned)(units < 65535 ? units : 65535));
  return cuda_ok(copy_vec_bytes(c) == 16
                     ? launch_dependent(fork_apply_kernel<uint4>, grid, kCopyThreads, 0, s, f, slabs, units)
                     : launch_dependent(fork_apply_kernel<uint2>, grid, kCopyThreads, 0, s, f, slabs, units),
                 "fork apply launch");
}

int launch_page_release(void *state, int *page_refs, const int *pages, int n, uint32_t *page_status, cudaStream_t s) {
  const ReleaseArgs r{state, page_refs, pages, n, page_status};
  if (n <= kReleaseOneBlock) {
    release_one_block_kernel<<<1, kAT, 0, s>>>(r);
    return cuda_ok(cudaGetLastError(), "page release launch");
  }
  const unsigned blocks = (unsigned)((n + 255LL) / 256);
  release_count_kernel<<<blocks, 256, 0, s>>>(r);
  int rc = cuda_ok(cudaGetLastError(), "page release launch (count)");
  if (rc) return rc;
  rc = cuda_ok(launch_dependent(release_sort_kernel, dim3(blocks), 256, 0, s, r), "page release launch (sort)");
  if (rc) return rc;
  return cuda_ok(launch_dependent(release_apply_kernel, dim3((unsigned)((n + (long long)kAT - 1) / kAT) + 1), kAT, 0, s, r),
                 "page release launch (apply)");
}

}  // namespace pfkv
