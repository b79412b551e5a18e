// prefix_attn.cu -- decode attention of a batch that shares long prefixes,
// each prefix read once for all its requests.
//
// For query row q of request b with prefix tokens t < T_g and its own tokens
// t >= T_g, softmax over both is joined from two partial results by the
// log-sum-exp rule:
//   M = max(m_1, m_2),  out = sum_i e^{m_i - M} o_i / sum_i e^{m_i - M} l_i,
// with m_i the maximum of the scaled scores of part i, l_i the sum of
// e^{z - m_i} and o_i the sum of e^{z - m_i} v.  Kernels, in one stream:
//   1. plan    one block per request: members of each group, lengths past
//              the prefix, the work line.
//   2. prefix  the groups' query rows as one matrix per KV head against the
//              prefix pages (prefix_kernel.cuh); beside it, on a spare warp,
//              the check that every member's first pages are the same pages
//              (and, under the tag check, are still its own).
//   3. split   each request's own pages: the grouped-query decode's split
//              kernel (decode_gqa.cuh) on lengths and tables past the prefix.
//   4. join    partial results of 2 and 3 to out; status.
#include <atomic>

#include "prefix_kernel.cuh"

namespace pfkv {

namespace {

// ---------------------------------------------------------------- plan

constexpr int kPlanThreads = 256;
constexpr int kPlanGroups = 64;  // groups whose segments block B keeps in shared memory

// Tokens of a prefix stay below this, so that a tile past the end still counts in int.
constexpr long long kMaxPrefixTokens = (1LL << 31) - 4096;

// Sum over the block (kPlanThreads threads); every thread gets it.
__device__ __forceinline__ int block_sum(int v, int *s_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if (lane == 0) s_sum[warp] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) s += s_sum[w];
  return s;
}

// Block b < B: request b.  Block B: the groups' segments of the work line.
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const PrefixArgs a) {
  // block B: requests of each group (low half: all, high half: those whose length covers the prefix), then the
  // first of the latter
  extern __shared__ uint32_t s_count[];
  __shared__ int s_sum[kPlanThreads / 32];
  __shared__ PrefixGroup s_groups[kPlanGroups];
  __shared__ PrefixHdr s_hdr;
  pdl_wait();
  pdl_launch_dependents();
  const int t = threadIdx.x, B = a.d.B, MP = a.d.MP, S = a.d.S;
  if ((int)blockIdx.x == B) {
    int *s_lead = reinterpret_cast<int *>(s_count + a.n_groups);
    for (int g = t; g < a.n_groups; g += kPlanThreads) {
      s_count[g] = 0u;
      s_lead[g] = B;
    }
    __syncthreads();
    for (int b = t; b < B; b += kPlanThreads) {
      const int g = a.group_of[b];
      if (g < 0 || g >= a.n_groups) continue;
      const long long L = a.d.seq_lens[b];
      const bool fits = L >= 1 && L <= (long long)MP * S && L >= (long long)a.group_pages[g] * S;
      atomicAdd(&s_count[g], fits ? 0x10001u : 1u);
      if (fits) atomicMin(&s_lead[g], b);
    }
    __syncthreads();
    if (t < 32) {  // 32 groups at a time, their sums carried along
      int first = 0, item = 0, longest = 0;
      long long unit = 0;
      for (int base = 0; base < a.n_groups; base += 32) {
        const int g = base + t;
        const uint32_t count = g < a.n_groups ? s_count[g] : 0u;
        const int all = (int)(count & 0xffffu), n = (int)(count >> 16);
        int pages = g < a.n_groups ? a.group_pages[g] : 0;
        // a bad one is reported by its requests
        if (pages < 0 || pages > MP || (long long)pages * S >= kMaxPrefixTokens || n == 0) pages = 0;
        longest = max(longest, pages);
        const HeadLine line = head_line(n, a.G, pages, a.c0);
        const int items = pages ? a.d.cache.num_kv_heads * line.blocks : 0;
        const long long units = pages ? a.d.cache.num_kv_heads * line.head : 0;
        int xn = all, xi = items;
        long long xu = units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int yn = __shfl_up_sync(0xffffffffu, xn, o), yi = __shfl_up_sync(0xffffffffu, xi, o);
          const long long yu = __shfl_up_sync(0xffffffffu, xu, o);
          if (t >= o) {
            xn += yn;
            xi += yi;
            xu += yu;
          }
        }
        const PrefixGroup pg{first + xn - all, n, g < a.n_groups ? s_lead[g] : 0, 0, pages, item + xi - items, unit + xu - units};
        if (g < kPlanGroups) s_groups[g] = pg;
        if (g < a.n_groups) a.groups[g] = pg;
        first += __shfl_sync(0xffffffffu, xn, 31);
        item += __shfl_sync(0xffffffffu, xi, 31);
        unit += __shfl_sync(0xffffffffu, xu, 31);
      }
      longest = __reduce_max_sync(0xffffffffu, longest);
      if (t == 0) {
        const long long r = unit / a.min_units;
        s_hdr = PrefixHdr{unit, unit == 0 ? 0 : r < 1 ? 1 : (int)(r < a.ctas ? r : a.ctas), longest};
        *a.hdr = s_hdr;
      }
    }
    __syncthreads();
    // the ranges' first pieces, a thread each
    const PrefixHdr hdr = s_hdr;
    for (int k = t; k < hdr.R; k += kPlanThreads) {
      PRange r;
      PWalk w{range_start(hdr, k), range_start(hdr, k + 1), k};
      r.item = PItem{};
      walk_next(a, a.n_groups <= kPlanGroups ? s_groups : a.groups, w, r.item);
      r.u = w.u;
      r.u1 = w.u1;
      a.ranges[k] = r;
    }
    return;
  }
  const int b = blockIdx.x;
  const int g = a.group_of[b], L = a.d.seq_lens[b];
  uint32_t bits = 0u;
  if (L < 1 || (long long)L > (long long)MP * S) bits |= PFKV_ST_BAD_LEN;
  if (g < -1 || g >= a.n_groups) bits |= PFKV_ST_BAD_GROUP;
  int pages = 0, rank = 0;
  if (g >= 0 && g < a.n_groups) {
    pages = a.group_pages[g];
    if (pages < 0 || pages > MP || (long long)pages * S >= kMaxPrefixTokens) {
      bits |= PFKV_ST_BAD_GROUP;
      pages = 0;
    }
    if (!bits && (long long)L < (long long)pages * S) bits |= PFKV_ST_BAD_LEN;
    // its place among all members, and in its group
    int before = 0, mine = 0;
    for (int k = t; k < B && !bits; k += kPlanThreads) {
      const int gk = a.group_of[k], Lk = a.d.seq_lens[k];
      before += gk >= 0 && gk < g;
      mine += gk == g && k < b && Lk >= 1 && (long long)Lk <= (long long)MP * S && (long long)Lk >= (long long)pages * S;
    }
    rank = block_sum(mine, s_sum);
    const int at = block_sum(before, s_sum) + rank;
    if (t == 0 && !bits) a.members[at] = b;
  }
  if (t == 0) {
    const long long own = (long long)L - (long long)pages * S;
    // a request that is already refused takes no further part
    a.own_len[b] = bits ? 0 : (int)own;
    a.skip[b] = pages;
    a.rank[b] = rank;
    // a new token belongs in a page of the request's own
    if (!bits && a.d.append && own == 0) bits |= PFKV_ST_BAD_LEN;
    a.pre_st[b] = bits;
    a.check_st[b] = 0u;
  }
}

// ---------------------------------------------------------------- join

// Per (request, query head): the pieces of the request's own pages (split
// kernel) and of its group's prefix, joined by the log-sum-exp rule.  Reads
// every partial once, a row of a piece per warp and load.  Bound by latency:
// a few dependent look-ups, then rows in flight.  kWarps warps share a row: one
// where there are rows enough to fill the SMs, eight (a block) for few rows
// of many pieces each.
constexpr int kJoinThreads = 256;
constexpr int kMaxJoin = 256 + 2 * kMaxRanges;
constexpr int kAhead = 6;  // rows a warp has in flight before it knows their weights

// A lane's share of the OR of n words (16-byte aligned, room for a multiple of four).
__device__ __forceinline__ int any_word(const int *words, int n, int lane) {
  int any = 0;
#pragma unroll 4
  for (int i = 4 * lane; i < n; i += 128) {
    const int4 v = *reinterpret_cast<const int4 *>(words + i);
    any |= v.x | (i + 1 < n ? v.y : 0) | (i + 2 < n ? v.z : 0) | (i + 3 < n ? v.w : 0);
  }
  return any;
}

template <int kD, int kWarps>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const PrefixArgs a) {
  constexpr int kCols = kD / 4, kPar = 32 / kCols;  // float4 columns; pieces a warp reads at once
  __shared__ float s_w[kWarps == 1 ? kJoinThreads / 32 : 1][kMaxJoin];
  __shared__ float4 s_acc[kWarps == 1 ? 1 : kWarps][32];
  pdl_wait();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const unsigned id = kWarps == 1 ? blockIdx.x * (kJoinThreads / 32) + warp : blockIdx.x;
  if (id >= (unsigned)a.d.B * (unsigned)a.d.Hq) return;  // kWarps 1 only: a whole warp, and no block barrier below
  const int b = (int)(id / (unsigned)a.d.Hq), hq = (int)(id - (unsigned)b * (unsigned)a.d.Hq);
  const int w0 = kWarps == 1 ? 0 : warp;  // this warp's place among the row's
  float *sw = s_w[kWarps == 1 ? warp : 0];
  // all that hangs on the request alone, at once
  const int own = a.own_len[b];
  const int count = a.d.split_count[b], first_piece = a.d.split_first[b];
  const uint32_t pre = a.pre_st[b];
  uint32_t st = pre | a.check_st[b];
  const PrefixRow pr = a.ctas > 0 ? a.rows[id] : PrefixRow{0, 0, 0, 0};
  // whether a CTA of either kernel gave up: four words a load, all of them on their way beside the rest
  int any = 0;
  if (hq == 0 && w0 == 0) {
    any |= any_word(a.d.cta_abort, a.d.n_ctas, lane);
    any |= any_word(a.aborts, a.ctas, lane);
  }
  // own pages
  int n_own = 0, c0 = 0;
  if (own > 0) {
    n_own = count;
    c0 = first_piece;
    if (n_own < 1 || n_own > a.d.max_splits || c0 < 0 || c0 > a.d.B * a.d.max_splits - n_own) {
      n_own = c0 = 0;  // a CTA of the split gave up before it wrote them
      st |= PFKV_ST_TIMEOUT;
    }
  }
  auto pre_row = [&](int i) {
    return (size_t)(pr.slot0 + (i >> pr.sh)) * kRows + pr.row + (pr.sh ? (i & 1) * (kRows / 2) : 0);
  };
  const int n = n_own + pr.n;
  // this warp's first rows, on their way beside the pieces' maxima
  const int col = lane % kCols, i0 = w0 * kPar + lane / kCols;
  auto row_of = [&](int i) {
    const float *src = i < n_own ? a.d.part_o + ((size_t)(c0 + i) * a.d.Hq + hq) * kD : a.o + pre_row(i - n_own) * kD;
    return __ldcg(reinterpret_cast<const float4 *>(src) + col);
  };
  float4 ahead[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = i0 + k * kWarps * kPar;
    ahead[k] = i < n ? row_of(i) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int i = lane; i < n_own * a.d.st_groups; i += 32) st |= a.d.part_st[(size_t)c0 * a.d.st_groups + i];
  // the pieces' maxima, then their weights
  auto ml_of = [&](int i) {
    return i < n_own ? a.d.part_ml[(size_t)(c0 + i) * a.d.Hq + hq] : a.ml[pre_row(i - n_own)];
  };
  const float2 ml0 = lane < n ? ml_of(lane) : make_float2(kNegInf, 0.f);  // the first 32 stay in registers
  float mx = ml0.x;
  for (int i = lane + 32; i < n; i += 32) mx = fmaxf(mx, ml_of(i).x);
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  st = __reduce_or_sync(0xffffffffu, st);
  float W = 0.f;
  for (int i = lane; i < n; i += 32) {
    const float2 ml = i < 32 ? ml0 : ml_of(i);
    const float w = fast_exp2(ml.x - mx);
    W += w * ml.y;
    if (w0 == 0) sw[i] = w;
  }
  for (int o = 16; o; o >>= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
  if (kWarps == 1) __syncwarp();
  else __syncthreads();
  if (hq == 0 && w0 == 0) {
    if (__any_sync(0xffffffffu, any != 0)) st |= PFKV_ST_TIMEOUT;
    if (lane == 0) a.d.status[b] = st;
  }
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (!st) {
    auto add = [&](float w, float4 v) {
      acc.x += w * v.x; acc.y += w * v.y; acc.z += w * v.z; acc.w += w * v.w;
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i0 + k * kWarps * kPar < n) add(sw[i0 + k * kWarps * kPar], ahead[k]);
#pragma unroll 8
    for (int i = i0 + kAhead * kWarps * kPar; i < n; i += kWarps * kPar) add(sw[i], row_of(i));
  }
  if (kPar == 2) {
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
  }
  if (kWarps > 1) {
    s_acc[kWarps == 1 ? 0 : warp][lane] = acc;
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int k = 1; k < kWarps; ++k) {
      const float4 v = s_acc[kWarps == 1 ? 0 : k][lane];
      acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
    }
  }
  if (lane >= kCols) return;
  const float inv = st ? 0.f : 1.f / W;
  acc.x *= inv; acc.y *= inv; acc.z *= inv; acc.w *= inv;
  const size_t at = (size_t)id * kCols + lane;
  if (a.out_bf16)
    reinterpret_cast<uint2 *>(a.d.out)[at] = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
  else
    reinterpret_cast<float4 *>(a.d.out)[at] = acc;
}

// ---------------------------------------------------------------- host side

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

struct PrefixLayout {
  size_t own_len, skip, pre_st, check_st, rank, members, groups, rows, hdr, ranges, ml, o, aborts, total;
};

// Slots: pieces of the work line, at most one per range and one per item more.
PrefixLayout prefix_layout(size_t first, int batch, int q_heads, int kv_heads, int dim, int n_groups) {
  const size_t B = (size_t)batch, G = (size_t)(q_heads / kv_heads);
  const size_t full = (size_t)n_groups < B ? (size_t)n_groups : B;  // groups that can have members
  const size_t items = (size_t)kv_heads * (B * G / kRows + full);
  const size_t slots = n_groups ? (items + kMaxRanges) * kRows : 0;
  PrefixLayout w;
  w.own_len = first;
  w.skip = w.own_len + up256(4 * B);
  w.pre_st = w.skip + up256(4 * B);
  w.check_st = w.pre_st + up256(4 * B);
  w.rank = w.check_st + up256(4 * B);
  w.members = w.rank + up256(4 * B);
  w.groups = w.members + up256(4 * B);
  w.rows = w.groups + up256(sizeof(PrefixGroup) * (size_t)n_groups);
  w.hdr = w.rows + (n_groups ? up256(sizeof(PrefixRow) * B * (size_t)q_heads) : 0);
  w.ranges = w.hdr + up256(sizeof(PrefixHdr));
  w.aborts = w.ranges + up256(sizeof(PRange) * kMaxRanges);
  w.ml = w.aborts + up256(4 * (size_t)kMaxRanges);
  w.o = w.ml + up256(sizeof(float2) * slots);
  w.total = w.o + up256(sizeof(float) * slots * dim);
  return w;
}

// A BF16 pool in boxes of 16 tokens x 64 values, as operand tiles hold them.
int make_tile_map(CUtensorMap *map, const void *pool, const DecodeArgs &d) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return cuda_fail(cudaErrorNotSupported, "cuTensorMapEncodeTiled entry point");
  const cuuint64_t row = 2ull * d.D;
  const cuuint64_t dims[4] = {(cuuint64_t)d.D, (cuuint64_t)d.S, (cuuint64_t)d.cache.num_kv_heads, (cuuint64_t)d.P};
  const cuuint64_t strides[3] = {row, row * d.S, row * d.S * d.cache.num_kv_heads};
  const cuuint32_t box[4] = {64, 16, 1, 1}, estr[4] = {1, 1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(pool), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PFKV_OK : cuda_fail(cudaErrorInvalidValue, "cuTensorMapEncodeTiled");
}

template <bool kFp8, int kD, int kTerms, bool kToken>
int run_prefix(PrefixArgs a, cudaStream_t s) {
  using C = PCfg<kFp8, kD, kTerms>;
  a.ctas = a.n_groups == 0 ? 0 : num_sms() < kMaxRanges ? num_sms() : kMaxRanges;
  const LineUnits units = line_units(a.d.S);
  a.c0 = units.c0;
  a.min_units = units.min_units;
  // all that can be refused comes before the first launch
  DecodeArgs own = a.d;
  own.beside = a.ctas > 0;
  own.seq_lens = a.own_len;
  SplitLaunch split;
  int rc = prepare_gqa_split(own, split);
  if (rc) return rc;
  a.d.n_ctas = split.a.n_ctas;
  a.d.st_groups = split.a.st_groups;
  CUtensorMap map_k{}, map_v{};
  if (!kFp8 && a.ctas > 0) {
    rc = make_tile_map(&map_k, a.d.k_pool, a.d);
    if (!rc) rc = make_tile_map(&map_v, a.d.v_pool, a.d);
    if (rc) return rc;
  }
  int dev = 0;
  cudaGetDevice(&dev);
  static std::atomic<uint64_t> attr_set{0};  // devices whose shared-memory limit is raised
  if (dev >= 64 || !(attr_set.load() >> dev & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(prefix_kernel<kFp8, kD, kTerms, kToken>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kTotal);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(prefix kernel)");
    if (dev < 64) attr_set.fetch_or(1ull << dev);
  }
  rc = cuda_ok(launch_dependent(prefix_plan_kernel, dim3((unsigned)a.d.B + 1u), kPlanThreads, 8 * (size_t)a.n_groups, s,
                                a),
               "prefix plan launch");
  if (rc) return rc;
  if (a.ctas > 0) {
    rc = cuda_ok(launch_dependent(prefix_kernel<kFp8, kD, kTerms, kToken>, dim3(a.ctas), kPThreads, C::kTotal, s, map_k,
                                  map_v, a),
                 "prefix kernel launch");
    if (rc) return rc;
  }
  rc = launch_gqa_split(split, s);
  if (rc) return rc;
  // eight warps a row where one each would leave SMs idle
  const long long rows = (long long)a.d.B * a.d.Hq;
  const bool few = rows < 8LL * num_sms();
  const dim3 grid((unsigned)(few ? rows : (rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32)));
  return cuda_ok(few ? launch_dependent(prefix_join_kernel<kD, kJoinThreads / 32>, grid, kJoinThreads, 0, s, a)
                     : launch_dependent(prefix_join_kernel<kD, 1>, grid, kJoinThreads, 0, s, a),
                 "prefix join launch");
}

// How many 16-bit terms carry a probability.  FP8 caches (f16 products): one
// holds 11 bits, below the rounding of a bf16 output; two hold 22.  BF16
// caches (bf16 products) 8 bits a term: two for a bf16 output, three for fp32.
template <int kD>
int dispatch_prefix(const PrefixArgs &a, cudaStream_t s) {
  if (a.d.dtype != PFKV_DTYPE_FP8_E4M3)
    return a.out_bf16 ? run_prefix<false, kD, 2, false>(a, s) : run_prefix<false, kD, 3, false>(a, s);
  if (a.d.scale_mode == PFKV_SCALE_PER_TOKEN)
    return a.out_bf16 ? run_prefix<true, kD, 1, true>(a, s) : run_prefix<true, kD, 2, true>(a, s);
  return a.out_bf16 ? run_prefix<true, kD, 1, false>(a, s) : run_prefix<true, kD, 2, false>(a, s);
}

}  // namespace

size_t prefix_ws_bytes(size_t first, int batch, int q_heads, int kv_heads, int dim, int n_groups) {
  return prefix_layout(first, batch, q_heads, kv_heads, dim, n_groups).total;
}

int launch_prefix_decode(const DecodeArgs &d, size_t ws_first, uint8_t *ws, const int *group_of,
                         const int *group_pages, int n_groups, int out_bf16, cudaStream_t s) {
  PrefixArgs a{};
  a.d = d;
  a.G = d.G;
  a.group_of = group_of;
  a.group_pages = group_pages;
  a.n_groups = n_groups;
  a.out_bf16 = out_bf16;
  const PrefixLayout L = prefix_layout(ws_first, d.B, d.Hq, d.cache.num_kv_heads, d.D, n_groups);
  a.own_len = reinterpret_cast<int *>(ws + L.own_len);
  a.skip = reinterpret_cast<int *>(ws + L.skip);
  a.pre_st = reinterpret_cast<uint32_t *>(ws + L.pre_st);
  a.check_st = reinterpret_cast<uint32_t *>(ws + L.check_st);
  a.rank = reinterpret_cast<int *>(ws + L.rank);
  a.members = reinterpret_cast<int *>(ws + L.members);
  a.groups = reinterpret_cast<PrefixGroup *>(ws + L.groups);
  a.rows = reinterpret_cast<PrefixRow *>(ws + L.rows);
  a.hdr = reinterpret_cast<PrefixHdr *>(ws + L.hdr);
  a.ranges = reinterpret_cast<PRange *>(ws + L.ranges);
  a.aborts = reinterpret_cast<int *>(ws + L.aborts);
  a.ml = reinterpret_cast<float2 *>(ws + L.ml);
  a.o = reinterpret_cast<float *>(ws + L.o);
  a.d.skip = a.skip;
  return d.D == 128 ? dispatch_prefix<128>(a, s) : dispatch_prefix<64>(a, s);
}

}  // namespace pfkv
