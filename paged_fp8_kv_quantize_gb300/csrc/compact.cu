// compact.cu -- closes the holes of a page pool: held pages with the highest
// ids move into the lowest free pages until the held pages are 0 .. held - 1
// (or a bound on the moves is reached), and the mappings follow.
//
// With H pages held, the m-th highest held page moves to the m-th lowest free
// one, for as long as the former's id is at least H.  Number the pages from
// the top, q = P - 1 - p, and let f(q) be the number of free pages before q.
// Then everything that is needed comes from one scan of the free flags:
//   a held page is move number q - f(q) as a source,
//   a free page is move number F - f(q) - 1 as a destination (F free pages),
//   and after m moves a page's place in the re-sorted free stack is q where
//   fewer than m held pages lie above it, f(q) + m for the other free pages.
// Two launches work this out (count per chunk, whose last block to finish scans
// the counts; plan: pools reach millions of pages) and a third moves the data,
// which is all that costs:
// it is bound by HBM, one read and one write of the moved pages.  In the same
// launch the held flags and holder counts follow, and every live table entry
// that names a moved page (found by a binary search of the sources, which
// the plan leaves in decreasing order) gets the page's new id and tag.
#include "alloc_state.cuh"
#include "page_copy.cuh"
#include "pfkv_device.cuh"

namespace pfkv {

namespace {

struct CompactArgs {
  void *state;
  uint32_t *page_tags;
  int *page_refs;  // NULL: not kept
  pfkv_cache c;
  int *table;
  uint32_t *tags;   // NULL: not kept
  const int *used;  // NULL: every entry is live
  int batch, MP;
  int max_moves;
  int *moved_src, *moved_dst, *n_moved;
};

// Chunk c covers q in [c * kAT, (c + 1) * kAT).
__global__ void __launch_bounds__(kAT) compact_count_kernel(const CompactArgs a) {
  __shared__ int s_last;
  __shared__ int s_warp[33];
  AllocView v = view(a.state);
  const int P = v.hdr->num_pages, n_chunks = gridDim.x;
  if (P != a.c.num_pages) {  // not this cache's allocator: nothing moves
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.n_moved = 0;
    return;
  }
  const long long q = (long long)blockIdx.x * kAT + threadIdx.x;
  const int n = __syncthreads_count(q < P && !v.held[P - 1 - q]);
  if (threadIdx.x == 0) {
    v.counts[blockIdx.x] = n;
    __threadfence();
    s_last = atomicAdd(&v.hdr->ticket, 1) == n_chunks - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  // the last block: exclusive scan of the chunks' counts
  if (threadIdx.x == 0) v.hdr->ticket = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int carry = 0;
  for (int base = 0; base < n_chunks; base += kAT) {
    const int c = base + (int)threadIdx.x;
    const int cnt = c < n_chunks ? __ldcg(&v.counts[c]) : 0;
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
    if (c < n_chunks) v.counts[c] = carry + s_warp[warp] + incl - cnt;
    carry += s_warp[32];
    __syncthreads();
  }
}

// The moves, the free stack after them and the destinations' new tags.
__global__ void __launch_bounds__(kAT) compact_plan_kernel(const CompactArgs a) {
  __shared__ int s_warp[33];
  pdl_wait();
  AllocView v = view(a.state);
  const int P = v.hdr->num_pages, F = v.hdr->free_count;
  if (P != a.c.num_pages) return;
  // moves: the free pages below H = P - F, which are those from q = F on
  int moves = 0;
  if (F > 0 && F < P) {
    const int cb = F / kAT;
    const long long qb = (long long)cb * kAT + threadIdx.x;
    const int before = v.counts[cb] + __syncthreads_count(qb < F && !v.held[P - 1 - qb]);
    moves = min(F - before, a.max_moves);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.n_moved = moves;
  const long long q = (long long)blockIdx.x * kAT + threadIdx.x;
  const bool in = q < P;
  const int p = (int)(P - 1 - q);
  const bool is_free = in && !v.held[p];
  int total;
  const int f = v.counts[blockIdx.x] + block_rank(is_free, s_warp, &total);
  if (!in) return;
  const int above = (int)q - f;  // held pages above p
  if (above < moves) {
    v.stack[q] = p;
    if (!is_free) a.moved_src[above] = p;
  } else if (is_free) {
    const int r = F - f - 1;
    if (r < moves) {
      a.moved_dst[r] = p;
      a.page_tags[p] += 1u;
    } else {
      v.stack[f + moves] = p;
    }
  }
}

constexpr int kTableEntries = 4 * kCopyThreads;  // table entries per unit

// Units, walked by the whole grid: ranges of the table, ranges of the moves
// (their flags and counts), then slabs of the moved pages.
template <typename V>
__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(const CompactArgs a, long long n_slabs) {
  pdl_wait();
  const int m = *a.n_moved, t = threadIdx.x;
  if (m == 0) return;
  AllocView v = view(a.state);
  const int lowest = a.moved_src[m - 1], P = a.c.num_pages;
  const long long entries = (long long)a.batch * a.MP;
  const long long tables = (entries + kTableEntries - 1) / kTableEntries;
  const long long pairs = (m + kCopyThreads - 1) / kCopyThreads;
  const long long units = tables + pairs + (long long)m * n_slabs;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    if (u < tables) {
      for (int j = 0; j < 4; ++j) {
        const long long e = u * kTableEntries + j * kCopyThreads + t;
        if (e >= entries) break;
        const int p = a.table[e];
        if (p < lowest || p >= P) continue;
        if (a.used) {
          const long long b = e / a.MP;
          if (e - b * a.MP >= a.used[b]) continue;
        }
        int lo = 0, hi = m - 1;  // moved_src decreases
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (a.moved_src[mid] > p) lo = mid + 1;
          else hi = mid;
        }
        if (a.moved_src[lo] != p) continue;  // a free page: a stale mapping
        if (a.tags) {
          if (a.tags[e] != a.page_tags[p]) continue;  // a stale mapping stays one
          a.tags[e] = a.page_tags[a.moved_dst[lo]];
        }
        a.table[e] = a.moved_dst[lo];
      }
    } else if (u < tables + pairs) {
      const long long r = (u - tables) * kCopyThreads + t;
      if (r < m) {
        const int src = a.moved_src[r], dst = a.moved_dst[r];
        v.held[src] = 0;
        v.held[dst] = 1;
        if (a.page_refs) {
          a.page_refs[dst] = a.page_refs[src];
          a.page_refs[src] = 0;
        }
      }
    } else {
      const long long w = u - tables - pairs;
      const long long r = w / n_slabs;
      copy_page_slab<V>(a.c, a.moved_src[r], a.moved_dst[r], a.c.page_size, w - r * n_slabs);
    }
  }
}

}  // namespace

int launch_page_compact(void *state, uint32_t *page_tags, int *page_refs, const pfkv_cache &c, int *block_table,
                        uint32_t *block_tags, const int *used, int batch, int max_pages, int max_moves,
                        int *moved_src, int *moved_dst, int *n_moved, cudaStream_t s) {
  const CompactArgs a{state, page_tags, page_refs, c,         block_table, block_tags, used, batch,
                      max_pages, max_moves, moved_src, moved_dst, n_moved};
  const int n_chunks = (int)((c.num_pages + (long long)kAT - 1) / kAT);
  compact_count_kernel<<<n_chunks, kAT, 0, s>>>(a);
  int rc = cuda_ok(cudaGetLastError(), "compact launch (count)");
  if (rc) return rc;
  rc = cuda_ok(launch_dependent(compact_plan_kernel, dim3(n_chunks), kAT, 0, s, a), "compact launch (plan)");
  if (rc) return rc;
  const long long slabs = copy_slabs(c);
  const long long entries = (long long)batch * max_pages;
  const long long moves = max_moves < c.num_pages / 2 ? max_moves : c.num_pages / 2;
  long long units = (entries + kTableEntries - 1) / kTableEntries + (moves + kCopyThreads - 1) / kCopyThreads;
  const long long cap = 8LL * num_sms();  // resident blocks
  units = moves > cap / slabs ? cap : units + moves * slabs;
  const unsigned grid = (unsigned)(units < 1 ? 1 : units < cap ? units : cap);
  return cuda_ok(copy_vec_bytes(c) == 16 ? launch_dependent(compact_move_kernel<uint4>, dim3(grid), kCopyThreads, 0, s, a, slabs)
                                         : launch_dependent(compact_move_kernel<uint2>, dim3(grid), kCopyThreads, 0, s, a, slabs),
                 "compact launch (move)");
}

}  // namespace pfkv
