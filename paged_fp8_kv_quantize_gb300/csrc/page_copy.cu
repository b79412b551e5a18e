// page_copy.cu -- copies pages of a paged cache to other pages of it: every
// head's first `slots` rows of K and V, bit for bit, and in per-token mode
// their scales.
//
// What it cannot do without is one read and one write of the copied bytes, so
// it is bound by HBM: no arithmetic, 16-byte loads and stores, one block per
// 16 KB slab of a page (page_copy.cuh).
#include "page_copy.cuh"

namespace pfkv {

namespace {

template <typename V>
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(pfkv_cache c, const int *src_pages,
                                                                 const int *dst_pages, const int *slots, int n_slabs,
                                                                 uint32_t *page_status) {
  const int i = blockIdx.x / n_slabs, slab = blockIdx.x - i * n_slabs;
  const int sp = src_pages[i], dp = dst_pages[i];
  const int n = slots ? slots[i] : c.page_size;
  uint32_t st = 0u;
  if (sp < 0 || sp >= c.num_pages || dp < 0 || dp >= c.num_pages) st |= PFKV_ST_PAGE_OOB;
  if (n < 0 || n > c.page_size) st |= PFKV_ST_BAD_LEN;
  if (slab == 0 && threadIdx.x == 0) page_status[i] = st;
  if (st || n == 0 || sp == dp) return;
  copy_page_slab<V>(c, sp, dp, n, slab);
}

}  // namespace

int launch_page_copy(const pfkv_cache &c, const int *src_pages, const int *dst_pages, const int *slots, int n_pages,
                     uint32_t *page_status, cudaStream_t s) {
  const long long slabs = copy_slabs(c);
  if (slabs > 0x7fffffffLL / n_pages) return PFKV_ERR_SHAPE;
  const unsigned grid = (unsigned)(slabs * n_pages);
  if (copy_vec_bytes(c) == 16)
    page_copy_kernel<uint4><<<grid, kCopyThreads, 0, s>>>(c, src_pages, dst_pages, slots, (int)slabs, page_status);
  else
    page_copy_kernel<uint2><<<grid, kCopyThreads, 0, s>>>(c, src_pages, dst_pages, slots, (int)slabs, page_status);
  return cuda_ok(cudaGetLastError(), "page copy launch");
}

}  // namespace pfkv
