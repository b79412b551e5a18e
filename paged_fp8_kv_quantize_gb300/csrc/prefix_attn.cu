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
//              the prefix, and the check that every member's first pages are
//              the same pages (and, under the tag check, are still its own).
//   2. prefix  the groups' query rows as one matrix per KV head against the
//              prefix pages (matrix instructions; see prefix_kernel).
//   3. split   each request's own pages: the grouped-query decode's split
//              kernel (decode_gqa.cu) on lengths and tables past the prefix.
//   4. join    partial results of 2 and 3 to out; status.
#include "prefix.cuh"

namespace pfkv {

namespace {

// ---------------------------------------------------------------- plan

constexpr int kPlanThreads = 256;

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
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const PrefixArgs a, const int rows) {
  extern __shared__ int s_count[];  // block B: requests of each group
  __shared__ int s_sum[kPlanThreads / 32];
  __shared__ int s_lead;
  __shared__ uint32_t s_bits;
  pdl_wait();
  const int t = threadIdx.x, B = a.d.B, MP = a.d.MP, S = a.d.S;
  if ((int)blockIdx.x == B) {
    for (int g = t; g < a.n_groups; g += kPlanThreads) s_count[g] = 0;
    __syncthreads();
    for (int b = t; b < B; b += kPlanThreads) {
      const int g = a.group_of[b];
      if (g >= 0 && g < a.n_groups) atomicAdd(&s_count[g], 1);
    }
    __syncthreads();
    if (t < 32) {  // 32 groups at a time, their sums carried along
      int first = 0, item = 0;
      long long unit = 0;
      for (int base = 0; base < a.n_groups; base += 32) {
        const int g = base + t;
        const int n = g < a.n_groups ? s_count[g] : 0;
        int pages = g < a.n_groups ? a.group_pages[g] : 0;
        if (pages < 0 || pages > MP || n == 0) pages = 0;  // a bad one is reported by its requests
        const int items = pages ? a.d.cache.num_kv_heads * row_blocks(n, a.G, rows) : 0;
        const long long units = (long long)items * pages;
        int xn = n, xi = items;
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
        if (g < a.n_groups) a.groups[g] = PrefixGroup{first + xn - n, n, pages, item + xi - items, unit + xu - units};
        first += __shfl_sync(0xffffffffu, xn, 31);
        item += __shfl_sync(0xffffffffu, xi, 31);
        unit += __shfl_sync(0xffffffffu, xu, 31);
      }
      if (t == 0) {
        const long long r = (unit + a.min_pages - 1) / a.min_pages;
        a.hdr->T = unit;
        a.hdr->R = (int)(r < a.ctas ? r : a.ctas);
      }
    }
    return;
  }
  const int b = blockIdx.x;
  const int g = a.group_of[b], L = a.d.seq_lens[b];
  uint32_t bits = 0u;
  if (L < 1 || (long long)L > (long long)MP * S) bits |= PFKV_ST_BAD_LEN;
  if (g < -1 || g >= a.n_groups) bits |= PFKV_ST_BAD_GROUP;
  int pages = 0;
  const bool member = g >= 0 && g < a.n_groups;
  if (member) {
    pages = a.group_pages[g];
    if (pages < 0 || pages > MP) {
      bits |= PFKV_ST_BAD_GROUP;
      pages = 0;
    }
    // place among all members, place in the group, the group's first request
    if (t == 0) {
      s_lead = b;
      s_bits = 0u;
    }
    __syncthreads();
    int before = 0, mine = 0;
    for (int k = t; k < B; k += kPlanThreads) {
      const int gk = a.group_of[k];
      before += gk >= 0 && gk < g;
      if (gk == g && k < b) {
        ++mine;
        atomicMin(&s_lead, k);
      }
    }
    const int rank = block_sum(mine, s_sum);
    const int at = block_sum(before, s_sum) + rank;
    const int lead = s_lead;
    if (t == 0) {
      a.rank[b] = rank;
      a.members[at] = b;
    }
    if (!bits && (long long)L < (long long)pages * S) bits |= PFKV_ST_BAD_LEN;
    uint32_t mb = 0u;
    if (!bits) {
      const int *row = a.d.block_table + (size_t)b * MP, *first = a.d.block_table + (size_t)lead * MP;
      const uint32_t *want = a.d.block_tags + (size_t)b * MP;  // read under the tag check only
#pragma unroll 4
      for (int i = t; i < pages; i += kPlanThreads) {
        const int p = row[i];
        if (p < 0 || p >= a.d.P)
          mb |= PFKV_ST_PAGE_OOB;
        else if ((a.d.flags & PFKV_FLAG_TAG_CHECK) && a.d.page_tags[p] != want[i])
          mb |= PFKV_ST_STALE_TAG;
        if (p != first[i]) mb |= PFKV_ST_PREFIX_DIFFERS;
      }
    }
    if (mb) atomicOr(&s_bits, mb);
    __syncthreads();
    bits |= s_bits;
  }
  if (t == 0) {
    const long long own = (long long)L - (long long)pages * S;
    // a request that is already refused takes no further part
    a.own_len[b] = bits ? 0 : (int)own;
    a.skip[b] = pages;
    // a new token belongs in a page of the request's own
    if (!bits && a.d.append && own == 0) bits |= PFKV_ST_BAD_LEN;
    a.pre_st[b] = bits;
  }
}

// ---------------------------------------------------------------- prefix, register-operand matrix instructions

constexpr int kRows = 128;    // rows of an item
constexpr int kTile = 64;     // tokens at a time
constexpr int kPThreads = 256;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// kTerms: 16-bit terms that carry a probability.  FP8 caches (f16 products):
// one term holds 11 bits, below the rounding of a bf16 output; two hold 22.
// BF16 caches (bf16 products): 8 bits a term; two for a bf16 output, three
// for an fp32 one.
template <bool kFp8, int kD, int kTerms>
__global__ void __launch_bounds__(kPThreads, 1) prefix_kernel(const PrefixArgs a) {
  constexpr int kStride = kD + 8;  // halves per row of a tile: rows 16 bytes apart modulo 128
  constexpr float kPScale = kFp8 ? 16384.f : 1.f;  // keeps small probabilities normal in f16
  __shared__ __align__(16) uint16_t s_k[kTile * kStride], s_v[kTile * kStride];
  __shared__ float s_ks[kTile], s_vs[kTile];
  pdl_wait();
  pdl_launch_dependents();
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, gid = lane >> 2, tq = lane & 3;
  const PrefixHdr hdr = *a.hdr;
  const int kr = blockIdx.x;
  if (t == 0) a.aborts[kr] = 0;
  if (kr >= hdr.R) return;
  const bool per_token = kFp8 && a.d.scale_mode == PFKV_SCALE_PER_TOKEN;
  const int S = a.d.S, H = a.d.cache.num_kv_heads;
  const long long u1 = range_start(hdr, kr + 1);
  for (long long u = range_start(hdr, kr); u < u1;) {
    int lo = 0, hi = a.n_groups - 1;  // the last group that starts at or before u
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.groups[mid].unit0 <= u) lo = mid;
      else hi = mid - 1;
    }
    const PrefixGroup g = a.groups[lo];
    const int item = (int)((u - g.unit0) / g.pages);
    const int p0 = (int)(u - g.unit0 - (long long)item * g.pages);
    const int p1 = (int)(u1 - u < g.pages - p0 ? p0 + (u1 - u) : g.pages);
    const int mb = row_blocks(g.n, a.G, kRows);
    const int h = item / mb, row0 = (item - h * mb) * kRows;
    const int n_rows = min(kRows, g.n * a.G - row0);
    const size_t slot = (size_t)kr + g.item0 + item;
    u += p1 - p0;
    const int *trow = a.d.block_table + (size_t)a.members[g.first] * a.d.MP;
    // this warp's 16 rows as A fragments; f16: row scaled by 2^e into [2^14, 2^15), exact
    uint32_t qf[kD / 16][4];
    float mult[2];
    float base = a.d.sm_scale_log2;
    if (kFp8 && !per_token) base *= a.d.k_scale[h];
    const bool busy = warp * 16 < n_rows;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = warp * 16 + gid + 8 * r;
      const uint16_t *src = nullptr;
      if (row < n_rows) {
        const int b = a.members[g.first + (row0 + row) / a.G];
        src = reinterpret_cast<const uint16_t *>(a.d.q) + ((size_t)b * a.d.Hq + h * a.G + (row0 + row) % a.G) * kD;
      }
      float mx = 0.f;
#pragma unroll
      for (int s = 0; s < kD / 16; ++s)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t w = src ? *reinterpret_cast<const uint32_t *>(src + 16 * s + 8 * c + 2 * tq) : 0u;
          qf[s][2 * c + r] = w;
          mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xffff0000u))));
        }
      int e = 0;
      if constexpr (kFp8) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if (mx > 0.f) {
          int x;
          frexpf(mx, &x);
          e = 15 - x;
        }
#pragma unroll
        for (int s = 0; s < kD / 16; ++s)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t w = qf[s][2 * c + r];
            qf[s][2 * c + r] = pack_f16x2(ldexpf(__uint_as_float(w << 16), e), ldexpf(__uint_as_float(w & 0xffff0000u), e));
          }
      }
      mult[r] = ldexpf(base, -e);
    }
    float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};
    float o[kD / 8][4];
#pragma unroll
    for (int i = 0; i < kD / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float vref = 0.f;  // per-token mode: the largest value scale so far; o is in its units

    const int n_tok = (p1 - p0) * S;
    for (int t0 = 0; t0 < n_tok; t0 += kTile) {
      __syncthreads();
      // stage kTile tokens of K and V as 16-bit values
      constexpr int kChunks = kD / 8;  // chunks of eight values a row
      for (int i = t; i < 2 * kTile * kChunks; i += kPThreads) {
        const int part = i / (kTile * kChunks), j = i % (kTile * kChunks);
        const int tok = j / kChunks, c = j % kChunks;
        uint4 out = make_uint4(0u, 0u, 0u, 0u);
        const int pid = t0 + tok < n_tok ? trow[p0 + (t0 + tok) / S] : -1;
        const bool ok = pid >= 0 && pid < a.d.P;
        const size_t row = ((size_t)(ok ? pid : 0) * H + h) * S + (t0 + tok) % S;
        if (ok) {
          if constexpr (kFp8) {
            const uint2 w = *reinterpret_cast<const uint2 *>(
                reinterpret_cast<const uint8_t *>(part ? a.d.v_pool : a.d.k_pool) + row * kD + c * 8);
            e4m3x4_to_f16x4(w.x, out.x, out.y);
            e4m3x4_to_f16x4(w.y, out.z, out.w);
          } else {
            out = *reinterpret_cast<const uint4 *>(
                reinterpret_cast<const uint16_t *>(part ? a.d.v_pool : a.d.k_pool) + row * kD + c * 8);
          }
        }
        *reinterpret_cast<uint4 *>((part ? s_v : s_k) + tok * kStride + c * 8) = out;
        if (per_token && c == 0) (part ? s_vs : s_ks)[tok] = ok ? (part ? a.d.v_scale : a.d.k_scale)[row] : 0.f;
      }
      __syncthreads();
      if (!busy) continue;
      // S = Q K^T
      float z[kTile / 8][4];
#pragma unroll
      for (int j = 0; j < kTile / 8; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) z[j][c] = 0.f;
#pragma unroll
      for (int s = 0; s < kD / 16; ++s)
#pragma unroll
        for (int j = 0; j < kTile / 16; ++j) {
          uint32_t bf[4];
          // matrices: tokens 16j..+7 / +8..15, dims 16s..+7 / +8..15
          ldsm4(bf, smem_addr(s_k + (16 * j + (lane & 7) + 8 * (lane >> 4)) * kStride + 16 * s + 8 * ((lane >> 3) & 1)));
          if constexpr (kFp8) {
            mma_f16(z[2 * j], qf[s], bf[0], bf[1]);
            mma_f16(z[2 * j + 1], qf[s], bf[2], bf[3]);
          } else {
            mma_bf16(z[2 * j], qf[s], bf[0], bf[1]);
            mma_bf16(z[2 * j + 1], qf[s], bf[2], bf[3]);
          }
        }
      float mx[2] = {kNegInf, kNegInf};
#pragma unroll
      for (int j = 0; j < kTile / 8; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int tok = 8 * j + 2 * tq + (c & 1);
          float x = z[j][c] * mult[c >> 1];
          if (per_token) x *= s_ks[tok];
          z[j][c] = t0 + tok < n_tok ? x : kNegInf;
          mx[c >> 1] = fmaxf(mx[c >> 1], z[j][c]);
        }
      float al[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        const float mn = fmaxf(m[r], mx[r]);
        al[r] = fast_exp2(m[r] - mn);
        m[r] = mn;
        l[r] *= al[r];
      }
      float vfac = kPScale;
      if (per_token) {
        float vm = vref;
        for (int i = 0; i < kTile; ++i) vm = fmaxf(vm, s_vs[i]);
        if (vm > vref) {
          al[0] *= vref / vm;
          al[1] *= vref / vm;
          vref = vm;
        }
        vfac = vref > 0.f ? kPScale / vref : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kD / 8; ++i) {
        o[i][0] *= al[0]; o[i][1] *= al[0]; o[i][2] *= al[1]; o[i][3] *= al[1];
      }
#pragma unroll
      for (int j = 0; j < kTile / 8; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float p = fast_exp2(z[j][c] - m[c >> 1]);
          l[c >> 1] += p;
          z[j][c] = p * (per_token ? vfac * s_vs[8 * j + 2 * tq + (c & 1)] : vfac);
        }
      // O += P V
#pragma unroll
      for (int s = 0; s < kTile / 16; ++s) {
        uint32_t pf[kTerms][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float x0 = z[2 * s + (q >> 1)][2 * (q & 1)], x1 = z[2 * s + (q >> 1)][2 * (q & 1) + 1];
#pragma unroll
          for (int k = 0; k < kTerms; ++k) {
            if constexpr (kFp8) {
              pf[k][q] = pack_f16x2(x0, x1);
              const __half2 y = *reinterpret_cast<const __half2 *>(&pf[k][q]);
              x0 -= __low2float(y);
              x1 -= __high2float(y);
            } else {
              pf[k][q] = pack_bf16x2(x0, x1);
              x0 -= __uint_as_float(pf[k][q] << 16);
              x1 -= __uint_as_float(pf[k][q] & 0xffff0000u);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kD / 16; ++i) {
          uint32_t bf[4];
          ldsm4t(bf, smem_addr(s_v + (16 * s + (lane & 15)) * kStride + 16 * i + 8 * (lane >> 4)));
#pragma unroll
          for (int k = 0; k < kTerms; ++k) {
            if constexpr (kFp8) {
              mma_f16(o[2 * i], pf[k], bf[0], bf[1]);
              mma_f16(o[2 * i + 1], pf[k], bf[2], bf[3]);
            } else {
              mma_bf16(o[2 * i], pf[k], bf[0], bf[1]);
              mma_bf16(o[2 * i + 1], pf[k], bf[2], bf[3]);
            }
          }
        }
      }
    }
    // the piece's partial result
    float fac = 1.f / kPScale;
    if (kFp8) fac *= per_token ? vref : a.d.v_scale[h];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      const int row = warp * 16 + gid + 8 * r;
      if (row >= n_rows) continue;
      if (tq == 0) a.ml[slot * kRows + row] = make_float2(m[r], l[r]);
      float *dst = a.o + (slot * kRows + row) * kD + 2 * tq;
#pragma unroll
      for (int i = 0; i < kD / 8; ++i)
        *reinterpret_cast<float2 *>(dst + 8 * i) = make_float2(o[i][2 * r] * fac, o[i][2 * r + 1] * fac);
    }
  }
}

// ---------------------------------------------------------------- join

// One block per (request, query head): the pieces of the request's own pages
// (split kernel) and of its group's prefix, joined by the log-sum-exp rule.
// Reads every partial once; 4 (D 128) or 8 (D 64) pieces at a time.
constexpr int kJoinThreads = 128;
constexpr int kMaxJoin = 256 + kMaxRanges;

template <int kD>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const PrefixArgs a) {
  constexpr int kCols = kD / 4, kPar = kJoinThreads / kCols;
  __shared__ float s_w[kMaxJoin], s_l[kMaxJoin];
  __shared__ float4 s_acc[kJoinThreads];
  __shared__ float s_red[2][kJoinThreads / 32];
  pdl_wait();
  const int b = blockIdx.x / a.d.Hq, hq = blockIdx.x - b * a.d.Hq, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  uint32_t st = a.pre_st[b];
  // own pages
  int n_own = 0, c0 = 0;
  if (a.own_len[b] > 0) {
    n_own = a.d.split_count[b];
    c0 = a.d.split_first[b];
    if (n_own < 1 || n_own > a.d.max_splits || c0 < 0 || c0 > a.d.B * a.d.max_splits - n_own) {
      n_own = c0 = 0;  // a CTA of the split gave up before it wrote them
      st |= PFKV_ST_TIMEOUT;
    }
  }
  // prefix
  int n_pre = 0, row = 0;
  long long slot0 = 0;
  const int g = a.group_of[b];
  if (!a.pre_st[b] && g >= 0 && a.skip[b] > 0) {
    const PrefixHdr hdr = *a.hdr;
    const PrefixGroup gr = a.groups[g];
    const int r = a.rank[b] * a.G + hq % a.G, blk = r / kRows;
    const int item = hq / a.G * row_blocks(gr.n, a.G, kRows) + blk;
    const long long first = gr.unit0 + (long long)item * gr.pages;
    const int k0 = range_of(hdr, first);
    n_pre = range_of(hdr, first + gr.pages - 1) - k0 + 1;
    slot0 = (long long)k0 + gr.item0 + item;
    row = r - blk * kRows;
  }
  const int n = n_own + n_pre;
  uint32_t bits = 0u;
  for (int i = t; i < n_own * a.d.st_groups; i += kJoinThreads) bits |= a.d.part_st[(size_t)c0 * a.d.st_groups + i];
  int any = 0;
  if (hq == 0) {
    for (int i = t; i < a.d.n_ctas; i += kJoinThreads) any |= a.d.cta_abort[i];
    for (int i = t; i < a.ctas; i += kJoinThreads) any |= a.aborts[i];
  }
  float mx = kNegInf;
  for (int i = t; i < n; i += kJoinThreads) {
    const float2 ml = i < n_own ? a.d.part_ml[(size_t)(c0 + i) * a.d.Hq + hq] : a.ml[(slot0 + i - n_own) * kRows + row];
    s_w[i] = ml.x;
    s_l[i] = ml.y;
    mx = fmaxf(mx, ml.x);
  }
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) s_red[0][warp] = mx;
  if (__syncthreads_or(bits != 0u)) {  // rare: gather which bits
    __shared__ uint32_t s_bits;
    if (t == 0) s_bits = 0u;
    __syncthreads();
    if (bits) atomicOr(&s_bits, bits);
    __syncthreads();
    st |= s_bits;
  }
  if (hq == 0) {
    const bool gave_up = __syncthreads_or(any) != 0;
    if (t == 0) a.d.status[b] = st | (gave_up ? (uint32_t)PFKV_ST_TIMEOUT : 0u);
  }
  mx = fmaxf(fmaxf(s_red[0][0], s_red[0][1]), fmaxf(s_red[0][2], s_red[0][3]));
  float W = 0.f;
  for (int i = t; i < n; i += kJoinThreads) {
    const float w = fast_exp2(s_w[i] - mx);
    W += w * s_l[i];
    s_w[i] = w;
  }
  for (int o = 16; o; o >>= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
  if (lane == 0) s_red[1][warp] = W;
  __syncthreads();
  W = s_red[1][0] + s_red[1][1] + s_red[1][2] + s_red[1][3];
  const int col = t % kCols, par = t / kCols;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (!st) {
#pragma unroll 4
    for (int i = par; i < n; i += kPar) {
      const float *src = i < n_own ? a.d.part_o + ((size_t)(c0 + i) * a.d.Hq + hq) * kD
                                   : a.o + ((size_t)(slot0 + i - n_own) * kRows + row) * kD;
      const float4 v = __ldcg(reinterpret_cast<const float4 *>(src) + col);
      const float w = s_w[i];
      acc.x += w * v.x; acc.y += w * v.y; acc.z += w * v.z; acc.w += w * v.w;
    }
  }
  s_acc[t] = acc;
  __syncthreads();
  if (t < kCols) {
    for (int k = 1; k < kPar; ++k) {
      const float4 v = s_acc[t + k * kCols];
      acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
    }
    const float inv = st ? 0.f : 1.f / W;
    acc.x *= inv; acc.y *= inv; acc.z *= inv; acc.w *= inv;
    const size_t at = ((size_t)b * a.d.Hq + hq) * kCols + t;
    if (a.out_bf16)
      reinterpret_cast<uint2 *>(a.d.out)[at] = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    else
      reinterpret_cast<float4 *>(a.d.out)[at] = acc;
  }
}

// ---------------------------------------------------------------- host side

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

struct PrefixLayout {
  size_t own_len, skip, pre_st, rank, members, groups, hdr, ml, o, aborts, total;
};

// Slots: pieces of the work line, at most one per range and one per item more.
PrefixLayout prefix_layout(size_t first, int batch, int q_heads, int kv_heads, int dim, int n_groups) {
  const size_t B = (size_t)batch, G = (size_t)(q_heads / kv_heads);
  const size_t full = (size_t)n_groups < B ? (size_t)n_groups : B;  // groups that can have members
  const size_t items = (size_t)kv_heads * (B * G / kRows + full);
  const size_t rows = n_groups ? (items + kMaxRanges) * kRows : 0;
  PrefixLayout w;
  w.own_len = first;
  w.skip = w.own_len + up256(4 * B);
  w.pre_st = w.skip + up256(4 * B);
  w.rank = w.pre_st + up256(4 * B);
  w.members = w.rank + up256(4 * B);
  w.groups = w.members + up256(4 * B);
  w.hdr = w.groups + up256(sizeof(PrefixGroup) * (size_t)n_groups);
  w.aborts = w.hdr + up256(sizeof(PrefixHdr));
  w.ml = w.aborts + up256(4 * (size_t)kMaxRanges);
  w.o = w.ml + up256(sizeof(float2) * rows);
  w.total = w.o + up256(sizeof(float) * rows * dim);
  return w;
}

template <bool kFp8, int kD, int kTerms>
int run_prefix(PrefixArgs a, cudaStream_t s) {
  a.ctas = num_sms() < kMaxRanges ? num_sms() : kMaxRanges;
  a.min_pages = (256 + a.d.S - 1) / a.d.S;
  int rc = cuda_ok(launch_dependent(prefix_plan_kernel, dim3((unsigned)a.d.B + 1u), kPlanThreads,
                                    4 * (size_t)a.n_groups, s, a, kRows),
                   "prefix plan launch");
  if (rc) return rc;
  rc = cuda_ok(launch_dependent(prefix_kernel<kFp8, kD, kTerms>, dim3(a.ctas), kPThreads, 0, s, a),
               "prefix kernel launch");
  if (rc) return rc;
  DecodeArgs own = a.d;
  own.seq_lens = a.own_len;
  rc = launch_gqa_split(own, s);
  if (rc) return rc;
  a.d.n_ctas = own.n_ctas;
  a.d.st_groups = own.st_groups;
  return cuda_ok(launch_dependent(prefix_join_kernel<kD>, dim3((unsigned)a.d.B * (unsigned)a.d.Hq), kJoinThreads, 0, s, a),
                 "prefix join launch");
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
  a.rank = reinterpret_cast<int *>(ws + L.rank);
  a.members = reinterpret_cast<int *>(ws + L.members);
  a.groups = reinterpret_cast<PrefixGroup *>(ws + L.groups);
  a.hdr = reinterpret_cast<PrefixHdr *>(ws + L.hdr);
  a.aborts = reinterpret_cast<int *>(ws + L.aborts);
  a.ml = reinterpret_cast<float2 *>(ws + L.ml);
  a.o = reinterpret_cast<float *>(ws + L.o);
  a.d.skip = a.skip;
  a.d.join = 1;
  const bool fp8 = d.dtype == PFKV_DTYPE_FP8_E4M3;
  if (d.D == 128) {
    if (fp8) return out_bf16 ? run_prefix<true, 128, 1>(a, s) : run_prefix<true, 128, 2>(a, s);
    return out_bf16 ? run_prefix<false, 128, 2>(a, s) : run_prefix<false, 128, 3>(a, s);
  }
  if (fp8) return out_bf16 ? run_prefix<true, 64, 1>(a, s) : run_prefix<true, 64, 2>(a, s);
  return out_bf16 ? run_prefix<false, 64, 2>(a, s) : run_prefix<false, 64, 3>(a, s);
}

}  // namespace pfkv
