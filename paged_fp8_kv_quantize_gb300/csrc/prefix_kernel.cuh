// prefix_kernel.cuh -- the groups' query rows against their shared pages, on
// the fifth-generation tensor cores (kernel 2 of prefix_attn.cu).
//
// One item is up to 256 query rows of one (group, KV head) over the group's
// pages, a piece a range of those pages; per unit of 128 rows and 64 tokens
//   S = Q K^T   (M = 128, N = 64, fp32 in tensor memory)
//   P = 2^(tau log2(e) S - m)
//   O += P V    (M = 128, N = head_dim; P from tensor memory)
// with 16-bit operands (f16 for an FP8 cache, whose codes convert exactly,
// bf16 for a BF16 one).  A probability is carried as kTerms 16-bit terms, each
// the rounding of what the terms before it leave; see prefix_attn.cu for how
// many a call takes.
//
// What bounds it: a KV byte of an FP8 cache meets 2 x rows products, so from
// about 150 rows on the tensor cores, not HBM.  Between a unit's products lies
// its softmax, whose latency (hand-over, tensor-memory reads and writes,
// exponentials) is longer than the products; so each row half keeps two score
// buffers, the next unit's QK^T runs while this one's softmax does, and PV
// follows when it can.  One CTA per SM:
//   warps 0-3, 4-7  softmax of row half 0 and 1: a thread owns a row, so that
//                   maxima and sums need no exchange; P overwrites S.
//   warps 8-11      FP8: operands e4m3 -> f16 from staged codes, once per CTA,
//                   into a ring of K and V tiles of 128 tokens in the 128-byte-
//                   swizzled layout; per-token scales parted between V operands
//                   and weights (hand_scales).  (BF16: the planner's tensor
//                   copies land in that ring by themselves.)
//   warps 12, 14    issue the MMAs of half 0 and 1.
//   warp 13         planner: works out the CTA's items and where each tile's
//                   rows lie (bounds-checked page ids), so that nobody else
//                   waits for a table entry, and issues the copies: FP8 codes
//                   into a staging ring (48 KB in flight and more), BF16
//                   tiles into the operand ring (64 KB and more).
//   warp 15         works out where the join finds each row's pieces and
//                   compares the requests' prefix pages, all CTAs together.
// An item of more than 128 rows has 128 in each half, over the same tokens.
// One of at most 128 rows gives both halves the same rows, half 0 the first 64
// tokens of each tile and half 1 the others; each half then leaves a partial
// result of its own.
//
// The running maximum m of a row is a reference that moves only when a weight
// would pass 2^14 (f16, where it still fits; 2^60 for bf16), which after the
// first units hardly happens; O is then rescaled in tensor memory by the row's
// own softmax warp, after the products it has handed over and before the next.
// f16 weights below 2^-14 are subnormal: off by at most 2^-25, alone or (second
// term) together, where the largest weight starts at 2^0 or, with two terms, at
// 2^10 (PCfg::kLead).
#pragma once

#include "prefix.cuh"

namespace pfkv {
namespace {

constexpr int kPThreads = 16 * 32;  // four warpgroups
constexpr int kItemSlots = 4;    // items announced ahead
constexpr int kTileSlots = 8;    // tiles announced ahead
// Registers a thread after the launch's 128: two softmax warpgroups, the
// operand warps, and the rest; 2 x 168 + 80 + 96 = 4 x 128.
constexpr int kRegsSoftmax = 168, kRegsLoader = 80, kRegsRest = 96;
static_assert(kRegsSoftmax >= 128 && kRegsLoader <= 128 && kRegsRest <= 128 &&
                  2 * kRegsSoftmax + kRegsLoader + kRegsRest <= 4 * 128,
              "an increase goes up and a decrease down, and all of them fit what the block was launched with");

// One tile, announced by the planner: the pool row of each 16 tokens' first
// one (they lie in one page), or -1 for tokens past the end or a page id
// outside the pool.
struct PTile {
  long long row[8];
  int kind;      // 0: ends the work, 1: a tile, 2: an item's first tile
  uint32_t rows; // bit g: row[g] is one
};
static_assert(sizeof(PTile) == 72, "tile slot");

constexpr int kTok = 128;  // tokens per tile

template <bool kFp8, int kD, int kTerms>
struct PCfg {
  static constexpr int kBufs = kTerms == 3 && kD == 128 ? 1 : 2;  // score buffers per half (tensor memory bounds it)
  // Rings as deep as shared memory allows.  (D 64 with 4 and 3 slots: two requests behind 65536 BF16 tokens 54.5 us
  // against 51.2, 64 behind FP8 ones with per-token scales 231 against 223; other FP8 calls the same.)
  static constexpr int kSlots = kD == 64 ? (kFp8 ? 6 : 8) : kFp8 ? 3 : 4;  // operand ring: K, V, K, V, ...
  static constexpr int kStage = !kFp8 ? 0 : kD == 64 ? 8 : 3;     // staged code tiles
  // Tiles whose per-token scales are kept: K's slot of tile n is free again when a product with the tile kSlots / 2
  // before it is done, which the softmax of the tile two before that precedes.
  static constexpr int kScaleSlots = kD == 64 ? 8 : 4;
  static constexpr uint32_t kBlk = 128 * 128;                     // 64 dims of a query half or of a tile
  static constexpr uint32_t kQBytes = kBlk * (kD / 64), kTBytes = kQBytes;
  static constexpr uint32_t kCodeBytes = kTok * kD;
  // tensor memory: score buffers (P lies over its scores), third terms, O
  __host__ __device__ static constexpr uint32_t col_s(int t, int b) { return (uint32_t)(t * kBufs + b) * 64; }
  __host__ __device__ static constexpr uint32_t col_x(int t, int b) { return 128 * kBufs + (uint32_t)(t * kBufs + b) * 32; }
  __host__ __device__ static constexpr uint32_t col_o(int t) { return 512 - (uint32_t)(2 - t) * kD; }
  static_assert((kTerms == 3 ? 192 : 128) * kBufs + 2 * kD <= 512, "tensor memory plan");
  // The maximum's weight is 2^kLead when a row's reference is set, and the
  // reference moves when a weight would pass 2^kGrow.  f16: weights up to
  // 2^14, times the rest of a V scale (below 2), stay below 65504,
  // and steps are 2^-24 at least, so a weight is off by 2^-25-kLead of the
  // largest; bf16 has the range of fp32.  A lead costs moves: 0.06 us a tile
  // (of 1.8) from 2^-4 to 2^0 with one term, up to 0.2 (of 2.4) from 2^0 to 2^10
  // with two.  Under a first token that takes 2^13 times a later one's weight (1024
  // tokens), the smallest lead put outputs off by 2e-2 and 5e-4 of sum p |v|;
  // these leave 2^-8, a bf16 output's rounding, and 3e-6.
  static constexpr float kLead = kFp8 && kTerms == 2 ? 10.f : 0.f, kGrow = kFp8 ? 14.f : 60.f;
  static constexpr uint32_t kOffQ = 0, kOffT = 2 * kQBytes, kOffCode = kOffT + kSlots * kTBytes;
  static constexpr uint32_t kOffCodeScale = kOffCode + kStage * kCodeBytes;  // K and V scales beside the codes of K
  static constexpr uint32_t kOffScale = kOffCodeScale + kStage * 2 * kTok * 4;
  static constexpr uint32_t kOffBars = kOffScale + (kFp8 ? kScaleSlots : 0) * (2 * kTok * 4 + 16);
  static constexpr uint32_t kOffItems = kOffBars + 8 * 96;
  static constexpr uint32_t kTotal = kOffItems + kItemSlots * sizeof(PItem) + kTileSlots * sizeof(PTile) + 1024;
  static constexpr uint32_t kIdQK = umma_idesc_f16(128, 64, !kFp8, 0, 0);
  static constexpr uint32_t kIdPV = umma_idesc_f16(128, kD, !kFp8, 0, 1);
  static_assert(kTotal <= 232448, "shared memory plan exceeds one SM");
};

constexpr int kMaxSlots = 8;
struct PBars {
  uint64_t *full, *empty;              // operand ring
  uint64_t *code_full, *code_empty;    // staging ring
  uint64_t *q_ready, *q_read;             // per half
  uint64_t *s_full, *p_full, *pv_done;    // per half and score buffer
  uint64_t *sc_full;                   // per-token scales
  uint64_t *item_full, *item_empty, *tile_full, *tile_empty;
  uint64_t *drain;  // one per issuing warp
};

__device__ __forceinline__ PBars pbars_at(uint8_t *base) {
  uint64_t *b = reinterpret_cast<uint64_t *>(base);
  PBars r;
  r.full = b; b += kMaxSlots;
  r.empty = b; b += kMaxSlots;
  r.code_full = b; b += kMaxSlots;
  r.code_empty = b; b += kMaxSlots;
  r.q_ready = b; b += 2;
  r.q_read = b; b += 2;
  r.s_full = b; b += 4;
  r.p_full = b; b += 4;
  r.pv_done = b; b += 4;
  r.sc_full = b; b += kMaxSlots;
  r.item_full = b; b += kItemSlots;
  r.item_empty = b; b += kItemSlots;
  r.tile_full = b; b += kTileSlots;
  r.tile_empty = b; b += kTileSlots;
  r.drain = b;
  return r;
}

__device__ __forceinline__ bool mbar_wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

// The new count must not be below (inc) or above (dec) the current one.
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// ---------------------------------------------------------------- planner (warp 13)

// Bulk copies of one staged tile (part 0: K, with the per-token scales of K
// and V; 1: V): lane g takes 16 tokens' codes, which are contiguous.
template <typename C, int kD, bool kToken>
__device__ __forceinline__ bool stage_codes(const PrefixArgs &a, uint8_t *smem, const PBars &B, const PTile &d,
                                            uint32_t rows, uint32_t i, int part, bool lead, uint64_t policy,
                                            volatile int *abort) {
  const int lane = threadIdx.x & 31;
  const uint32_t s = i % C::kStage;
  if (!mbar_wait_warp(&B.code_empty[s], ((i / C::kStage) & 1u) ^ 1u, abort)) return false;
  const uint32_t each = 16 * kD + (kToken && part == 0 ? 128 : 0);
  if (lead) mbar_arrive_expect_tx(&B.code_full[s], each * (uint32_t)__popc(rows));
  __syncwarp();
  if (rows >> lane & 1u) {
    const long long row = d.row[lane];
    const uint8_t *pool = static_cast<const uint8_t *>(part ? a.d.v_pool : a.d.k_pool);
    bulk_load_stream(smem + C::kOffCode + s * C::kCodeBytes + lane * 16 * kD, pool + row * kD, 16 * kD,
                     &B.code_full[s], policy);
    if (kToken && part == 0) {
      float *dst = reinterpret_cast<float *>(smem + C::kOffCodeScale) + s * 2 * kTok + 16 * lane;
      bulk_load_stream(dst, a.d.k_scale + row, 64, &B.code_full[s], policy);
      bulk_load_stream(dst + kTok, a.d.v_scale + row, 64, &B.code_full[s], policy);
    }
  }
  return true;
}

// BF16: tensor copies of tile i of the operand ring, 16 tokens x 64 values
// each, lane l % 8 the tokens and l / 8 the values.  Tokens without a row get
// the copy's fill value: a page past the pool's last reads as zeros.
template <typename C, int kD>
__device__ __forceinline__ bool copy_tile(const CUtensorMap &map, uint8_t *smem, const PBars &B, uint32_t i, int page,
                                          int slot, int h, bool live, bool lead, uint64_t policy, volatile int *abort) {
  const int lane = threadIdx.x & 31;
  const uint32_t s = i % C::kSlots;
  if (!mbar_wait_warp(&B.empty[s], ((i / C::kSlots) & 1u) ^ 1u, abort)) return false;
  if (lead) mbar_arrive_expect_tx(&B.full[s], C::kTBytes);
  __syncwarp();
  if (lane < kD / 8 && live)
    tma_load_4d_stream(smem + C::kOffT + s * C::kTBytes + (lane >> 3) * C::kBlk + (lane & 7) * 16 * 128, &map,
                       &B.full[s], (lane >> 3) * 64, slot, h, page, policy);
  return true;
}

template <bool kFp8, int kD, int kTerms, bool kToken>
__device__ __forceinline__ void plan_tiles(const PrefixArgs &a, const CUtensorMap &map_k, const CUtensorMap &map_v,
                                           uint8_t *smem, const PBars &B, volatile int *abort) {
  using C = PCfg<kFp8, kD, kTerms>;
  PItem *items = reinterpret_cast<PItem *>(smem + C::kOffItems);
  PTile *tiles = reinterpret_cast<PTile *>(smem + C::kOffItems + kItemSlots * sizeof(PItem));
  const int lane = threadIdx.x & 31, S = a.d.S, H = a.d.cache.num_kv_heads;
  const uint64_t policy = l2_evict_first_policy();
  constexpr int kGroups = kTok / 16, kAtOnce = 32 / kGroups;  // 16-token groups of a tile; tiles per look-up
  // the range's first piece comes from the plan: working it out here, in code that runs once and so out of a cold
  // instruction cache, took 3.4 us.  For the same reason the loop first goes over a tile that is none (live false),
  // while the plan is on its way: nothing is read, copied or announced (fp32 document 73.8 -> 71.7 us, its step with
  // bf16 output 106.4 -> 105.3).
  PItem first{};
  PWalk w{};
  uint32_t n = 0;
  bool ok = true, live = false, lead = false;  // lead: lane 0 of a live warp
  for (uint32_t i = 0; ok;) {
    PItem it{};
    if (i == 0) it = first;
    bool have = true;
    if (live) have = i == 0 ? it.n_rows != 0 : walk_next(a, a.groups, w, it);
    if (!mbar_wait_warp(&B.item_empty[i % kItemSlots], ((i / kItemSlots) & 1u) ^ 1u, abort)) break;
    if (lead) {
      items[i % kItemSlots] = it;
      mbar_arrive(&B.item_full[i % kItemSlots]);
    }
    const int n_look = live && have ? (it.p1 - it.p0) * S : 0, n_tok = max(n_look, 1);
    const int *trow = have ? a.d.block_table + (size_t)it.lead * a.d.MP + it.p0 : nullptr;
    auto look_up = [&](int t0) -> int {
      const int tok = t0 + 16 * lane;
      return tok < n_look ? __ldg(trow + tok / S) : -1;
    };
    int next = look_up(0);
    for (int t0 = 0; t0 < n_tok && ok; t0 += kAtOnce * kTok) {
      const int p = next;
      next = look_up(t0 + kAtOnce * kTok);  // on its way while this batch goes out
      const bool fine = p >= 0 && p < a.d.P;
      const uint32_t rows = __ballot_sync(0xffffffffu, fine);
      for (int k = 0; k < kAtOnce && t0 + k * kTok < n_tok; ++k, ++n) {
        if constexpr (!kFp8) {
          if (!have) return;
          const int g = kGroups * k + (lane & 7);
          const int page = __shfl_sync(0xffffffffu, fine ? p : a.d.P, g), slot = (t0 + 16 * g) % S;
          // test hook: the first CTA never gets its first tile, and the other warps' bounded waits give up
          if (live && (a.d.flags & PFKV_FLAG_TEST_WITHHOLD) && blockIdx.x == 0 && n == 0) return;
          ok = copy_tile<C, kD>(map_k, smem, B, 2 * n, page, slot, it.h, live, lead, policy, abort);
          ok = ok && copy_tile<C, kD>(map_v, smem, B, 2 * n + 1, page, slot, it.h, live, lead, policy, abort);
          if (!ok) break;
          continue;
        }
        PTile &d = tiles[n % kTileSlots];
        ok = mbar_wait_warp(&B.tile_empty[n % kTileSlots], ((n / kTileSlots) & 1u) ^ 1u, abort);
        if (!ok) break;
        if (lane / kGroups == k)
          d.row[lane % kGroups] = fine ? ((long long)p * H + it.h) * S + (t0 + 16 * lane) % S : -1;
        const uint32_t mine = rows >> (kGroups * k) & ((1u << kGroups) - 1u);
        if (lane == 0) {
          d.kind = !have ? 0 : t0 + k == 0 ? 2 : 1;
          d.rows = mine;
        }
        __syncwarp();
        if (lead) mbar_arrive(&B.tile_full[n % kTileSlots]);
        if constexpr (kFp8) {
          for (int part = 0; part < 2 && have && ok; ++part)
            ok = stage_codes<C, kD, kToken>(a, smem, B, d, mine, 2 * n + part, part, lead, policy, abort);
        }
        if (!ok) break;
      }
    }
    if (!have) return;
    if (live) {
      ++i;
      continue;
    }
    pdl_wait();
    pdl_launch_dependents();
    if ((int)blockIdx.x >= a.hdr->R) return;
    const PRange r = a.ranges[blockIdx.x];
    first = r.item;
    w = PWalk{r.u, r.u1, (int)blockIdx.x};
    live = true;
    lead = lane == 0;
    n = 0;
  }
  // a wait gave up: copies in flight land before the block may exit (waits of copies that were never issued, or that
  // a later one has overtaken, run out)
  constexpr uint32_t kRing = kFp8 ? C::kStage : C::kSlots;
  uint64_t *landed = kFp8 ? B.code_full : B.full;
  const uint32_t issued = 2 * n + 2;  // at most
  for (uint32_t i = issued > kRing + 2 ? issued - kRing - 2 : 0; i < issued; ++i) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(&landed[i % kRing], (i / kRing) & 1u))
      if (global_timer_ns() - t0 > kWaitLimitNs / 8) break;
  }
}

// ---------------------------------------------------------------- prefix check (warp 15)

// Every member's first pages are the group's (those of its first request), lie
// inside the pool and, under the tag check, have the tag of the member's
// mapping.  (Request, 512 pages) at a time, over all CTAs.
__device__ __forceinline__ void check_prefixes(const PrefixArgs &a, const PrefixHdr &hdr) {
  constexpr int kChunk = 512;
  const int lane = threadIdx.x & 31;
  const long long chunks = (hdr.max_pages + kChunk - 1) / kChunk;
  const bool tag_check = (a.d.flags & PFKV_FLAG_TAG_CHECK) != 0u;
  for (long long id = blockIdx.x; id < a.d.B * chunks; id += gridDim.x) {
    const int b = (int)(id / chunks), lo = (int)(id - b * chunks) * kChunk;
    if (a.pre_st[b] || lo >= a.skip[b]) continue;  // refused already, or no prefix there
    const int hi = min(lo + kChunk, a.skip[b]), lead = a.groups[a.group_of[b]].lead;
    const int *row = a.d.block_table + (size_t)b * a.d.MP, *first = a.d.block_table + (size_t)lead * a.d.MP;
    const uint32_t *want = a.d.block_tags + (size_t)b * a.d.MP;  // read under the tag check only
    uint32_t bits = 0u;
#pragma unroll 4
    for (int i = lo + lane; i < hi; i += 32) {
      const int p = row[i];
      if (p < 0 || p >= a.d.P) bits |= PFKV_ST_PAGE_OOB;
      else if (tag_check && a.d.page_tags[p] != want[i]) bits |= PFKV_ST_STALE_TAG;
      if (p != first[i]) bits |= PFKV_ST_PREFIX_DIFFERS;
    }
    if (bits) atomicOr(&a.check_st[b], bits);
  }
}

// Every row's pieces, for the join; rows spread over all CTAs.
__device__ __forceinline__ void find_pieces(const PrefixArgs &a, const PrefixHdr &hdr) {
  const unsigned all = (unsigned)a.d.B * (unsigned)a.d.Hq;
  for (unsigned id = blockIdx.x * 32 + (threadIdx.x & 31); id < all; id += gridDim.x * 32) {
    const int b = (int)(id / (unsigned)a.d.Hq), hq = (int)(id - (unsigned)b * (unsigned)a.d.Hq);
    PrefixRow pr{0, 0, 0, 0};
    if (!a.pre_st[b] && a.group_of[b] >= 0 && a.skip[b] > 0)
      pr = row_pieces(hdr, a.groups[a.group_of[b]], a.G, a.c0, a.rank[b], hq);
    a.rows[id] = pr;
  }
}

// ---------------------------------------------------------------- operands of FP8 caches (warps 8-11)

// Per-token scales of tile n, from beside its staged K codes.  K scales go to
// the softmax as they are.  A V scale is parted: a weight times the whole scale
// would leave f16's normal range wherever one token's scale is far above the
// others' (the scale of an all-zero row is 1), so its power of two goes into
// the token's V operand, as far as f16 holds every code exactly there
// (2^-14 .. 2^7), and the weight takes the rest, [1, 2) for scales within 2^18 of
// the largest:
//   scale = rest 2^shift 2^(ref - 134),  shift = clamp(e - ref + 7),
// with e a scale's biased exponent and ref a reference that starts 3 above the
// largest e of a tile and moves when one exceeds it (O is then rescaled).
// (A bf16 output behind an all-zero row, scale 1, among rows of 1e-3 at most
// was off by 2.9e-2 of its norm with the whole scale on the weight.)
// Every operand warp reads all of the tile's V scales for their maximum, so
// that the warps need not meet, and writes its own 32 tokens'.  shifts: byte i
// of lane r is shift + 15 of token 32 i + r.
constexpr int kRefSpare = 3, kRefLeast = 8;  // the least reference keeps 2^(ref - 134) a normal number
template <typename C>
__device__ __forceinline__ void hand_scales(uint8_t *smem, const PBars &B, uint32_t n, uint32_t stage, uint32_t rows,
                                            int &ref, uint32_t &shifts, int t) {
  float *dst = reinterpret_cast<float *>(smem + C::kOffScale) + (n % C::kScaleSlots) * (2 * kTok + 4);
  const float *src = reinterpret_cast<const float *>(smem + C::kOffCodeScale) + stage * 2 * kTok;
  const int lane = t & 31, warp = t >> 5;
  int e[kTok / 32], most = 0;
  float mine = 0.f;
#pragma unroll
  for (int i = 0; i < kTok / 32; ++i) {
    const int r = 32 * i + lane;
    const float v = rows >> (r >> 4) & 1u ? src[kTok + r] : 0.f;
    e[i] = (int)(__float_as_uint(v) >> 23 & 255u);
    most = max(most, e[i]);
    if (i == warp) mine = v;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (most > ref) ref = most + kRefSpare;
  shifts = 0u;
#pragma unroll
  for (int i = 0; i < kTok / 32; ++i) shifts |= (uint32_t)min(max(e[i] - ref + 22, 1), 22) << (8 * i);
  dst[t] = rows >> (t >> 4) & 1u ? src[t] : 0.f;
  // by 2^(134 - ref - shift) as two factors, either of which is a normal number
  const int by = 149 - ref - (int)(shifts >> (8 * warp) & 255u), half = by >> 1;
  auto pow2 = [](int k) { return __uint_as_float((uint32_t)(k + 127) << 23); };
  dst[kTok + t] = mine * pow2(half) * pow2(by - half);
  if (t == 0) dst[2 * kTok] = pow2(ref - 134);
  __syncwarp();
  if (lane == 0) mbar_arrive(&B.sc_full[n % C::kScaleSlots]);
}

// FP8: staged codes to f16 operands.  A thread takes 16 codes of a row at a
// time (8 lanes a row of 128, 4 of 64).
template <bool kFp8, int kD, int kTerms, bool kToken>
__device__ __forceinline__ void loader_fp8(const PrefixArgs &a, uint8_t *smem, const PBars &B, volatile int *abort) {
  using C = PCfg<kFp8, kD, kTerms>;
  constexpr int kLanes = kD / 16;                  // lanes a row
  constexpr int kRowsIt = 128 / kLanes;            // tokens per iteration
  constexpr int kIt = kTok / kRowsIt;
  static_assert(kTok == 128, "one token per operand thread for the scales");
  const PTile *tiles = reinterpret_cast<const PTile *>(smem + C::kOffItems + kItemSlots * sizeof(PItem));
  const int t = threadIdx.x - 8 * 32, lane = t & 31, c = t % kLanes;
  // D 128: the second half of a row goes with the first half of its neighbour, so that eight lanes' stores, which
  // the swizzle places by row and 16-byte chunk, meet different banks
  const int r_it = (t / kLanes) ^ (kD == 128 ? c >> 2 : 0);
  const uint32_t s_ring = smem_addr(smem + C::kOffT), s_code = smem_addr(smem + C::kOffCode) + r_it * kD + 16 * c;
  const bool withhold = (a.d.flags & PFKV_FLAG_TEST_WITHHOLD) && blockIdx.x == 0;
  int ref = kRefLeast;
  uint32_t shifts = 0u;
  for (uint32_t n = 0;; ++n) {
    if (!mbar_wait_warp(&B.tile_full[n % kTileSlots], (n / kTileSlots) & 1u, abort)) return;
    const int kind = tiles[n % kTileSlots].kind;
    const uint32_t rows = tiles[n % kTileSlots].rows;
    if (kind == 0) return;
    if (kind == 2) ref = kRefLeast;
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
      const uint32_t i = 2 * n + part, st = i % C::kStage, slot = i % C::kSlots;
      if (!mbar_wait_warp(&B.code_full[st], (i / C::kStage) & 1u, abort)) return;
      uint4 x[kIt];
#pragma unroll
      for (int k = 0; k < kIt; ++k) {
        const int r = k * kRowsIt + r_it;
        x[k] = lds128(s_code + st * C::kCodeBytes + k * kRowsIt * kD);
        // never copied: what stands there may be NaN
        if (rows != 0xffu && !(rows >> (r >> 4) & 1u)) x[k] = make_uint4(0u, 0u, 0u, 0u);
      }
      if (!mbar_wait_warp(&B.empty[slot], ((i / C::kSlots) & 1u) ^ 1u, abort)) return;
      if (kToken && part == 0) hand_scales<C>(smem, B, n, st, rows, ref, shifts, t);
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.code_empty[st]);
      const uint32_t base = s_ring + slot * C::kTBytes;
      // K as it is.  One code for both parts: a second copy of this loop cost more (instruction cache; document step
      // with bf16 output 133 us against 128) than the products by 1.
      const uint32_t by = part ? shifts : 0x0f0f0f0fu;
#pragma unroll
      for (int k = 0; k < kIt; ++k) {
        const int r = k * kRowsIt + r_it;
        uint4 lo, hi;
        e4m3x4_to_f16x4(x[k].x, lo.x, lo.y);
        e4m3x4_to_f16x4(x[k].y, lo.z, lo.w);
        e4m3x4_to_f16x4(x[k].z, hi.x, hi.y);
        e4m3x4_to_f16x4(x[k].w, hi.z, hi.w);
        if constexpr (kToken) {
          const uint32_t s4 = __shfl_sync(0xffffffffu, by, r & 31);
          const uint32_t f = (s4 >> (8 * (k * kRowsIt / 32)) & 255u) * 0x04000400u;  // 2^shift, twice; exact products
          lo.x = mul_f16x2(lo.x, f); lo.y = mul_f16x2(lo.y, f); lo.z = mul_f16x2(lo.z, f); lo.w = mul_f16x2(lo.w, f);
          hi.x = mul_f16x2(hi.x, f); hi.y = mul_f16x2(hi.y, f); hi.z = mul_f16x2(hi.z, f); hi.w = mul_f16x2(hi.w, f);
        }
        const uint32_t row = base + (c >> 2) * C::kBlk + r * 128;  // 16-byte chunks 2c and 2c + 1 of the row
        sts128(row + ((((2 * c) & 7) ^ (r & 7)) << 4), lo);
        sts128(row + ((((2 * c + 1) & 7) ^ (r & 7)) << 4), hi);
      }
      fence_async_smem();
      __syncwarp();
      // test hook: the first CTA never hands its first tile over, and the other warps' bounded waits give up
      if (withhold && i == 0) return;
      if (lane == 0) mbar_arrive(&B.full[slot]);
    }
    if (lane == 0) mbar_arrive(&B.tile_empty[n % kTileSlots]);
  }
}

// ---------------------------------------------------------------- MMA issuers (warps 12 and 14)

// The whole warp runs the loops and one elected lane issues: everything that an
// MMA takes is then the same in all lanes and lives in uniform registers.
// (With one thread running the loops, each MMA paid for moving its
// descriptors there: the document step took 117 us in this kernel.)
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e != 0;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Waits, bounded, until every MMA this thread issued has completed (before
// tensor memory is released).
__device__ __forceinline__ void drain_mmas(uint64_t *bar) {
  if (elect_one()) umma_commit(bar);
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, 0))
    if (global_timer_ns() - t0 > kWaitLimitNs) break;
}

// Tokens of item i and whether it is split; 0: no more work, or a wait gave up.
template <typename C>
__device__ __forceinline__ int next_item(uint8_t *smem, const PBars &B, uint32_t i, int S, bool &split,
                                         volatile int *abort) {
  if (!mbar_wait_warp(&B.item_full[i % kItemSlots], (i / kItemSlots) & 1u, abort)) return 0;
  const PItem &it = reinterpret_cast<const PItem *>(smem + C::kOffItems)[i % kItemSlots];
  const int n_tok = uniform(it.n_rows ? (it.p1 - it.p0) * S : 0);
  split = uniform(it.split) != 0;
  __syncwarp();
  if (elect_one()) mbar_arrive(&B.item_empty[i % kItemSlots]);
  return n_tok;
}

// Half t's products.  Unit v of an item is 64 of its tokens: QK^T of the first
// kBufs units, then for each unit PV, once P is in place, and the QK^T kBufs
// units further on into the score buffer that this PV reads P from.  MMAs that
// one thread issues execute in the order of issue, so that no wait lies between
// the two; and with a warp of its own a half that waits for a moved reference
// does not hold up the other.
template <bool kFp8, int kD, int kTerms>
__device__ __forceinline__ void issue_half(const PrefixArgs &a, uint8_t *smem, const PBars &B, uint32_t tmem, int t,
                                           volatile int *abort) {
  using C = PCfg<kFp8, kD, kTerms>;
  const uint64_t dq = umma_sdesc(smem_addr(smem + C::kOffQ) + t * C::kQBytes, 16, 1024, 2);
  const uint64_t dk = umma_sdesc(smem_addr(smem + C::kOffT), 16, 1024, 2);
  const uint64_t dv = umma_sdesc(smem_addr(smem + C::kOffT), C::kBlk, 1024, 2);
  const uint32_t s_col = tmem + C::col_s(0, 0) + (uint32_t)(t * C::kBufs) * 64;
  const uint32_t x_col = tmem + C::col_x(0, 0) + (uint32_t)(t * C::kBufs) * 32;
  const uint32_t o_col = tmem + C::col_o(0) + (uint32_t)t * kD;
  uint32_t tile0 = 0, u0 = 0;  // tiles, units before this item
  bool ok = true, split = false;
  for (uint32_t i = 0; ok; ++i) {
    const int n_tok = next_item<C>(smem, B, i, a.d.S, split, abort);
    if (n_tok == 0) break;
    const int tiles = (n_tok + kTok - 1) / kTok, chunks = (n_tok + 63) / 64;
    const int units = split ? (chunks - t + 1) / 2 : chunks;
    // tile of unit v, which 64 tokens of it, and whether the half is done with the tile then
    auto tile_of = [&](int v) { return split ? v : v >> 1; };
    auto part_of = [&](int v) { return split ? t : v & 1; };
    auto last_of = [&](int v) { return split || (v & 1) || v == units - 1; };
    auto slot_of = [&](int k, int part) { return (2 * (tile0 + (uint32_t)k) + (uint32_t)part) % C::kSlots; };
    auto wait_tile = [&](int k, int part) {
      const uint32_t j = 2 * (tile0 + (uint32_t)k) + (uint32_t)part;
      return mbar_wait_warp(&B.full[j % C::kSlots], (j / C::kSlots) & 1u, abort);
    };
    auto qk = [&](int v) {
      const int k = tile_of(v), c = part_of(v);
      if (split || !(v & 1)) {
        ok = wait_tile(k, 0);
        if (!ok) return;
        tc_fence_after();
      }
      const uint32_t slot = slot_of(k, 0), b = (u0 + (uint32_t)v) % C::kBufs;
      const uint64_t dks = dk + (uint64_t)((slot * C::kTBytes + c * 64 * 128) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int s = 0; s < kD / 16; ++s)
          umma_f16(s_col + 64 * b, dq + (uint64_t)(((s >> 2) * C::kBlk + (s & 3) * 32) >> 4),
                   dks + (uint64_t)(((s >> 2) * C::kBlk + (s & 3) * 32) >> 4), C::kIdQK, s ? 1u : 0u);
        umma_commit(&B.s_full[2 * t + b]);
        if (last_of(v)) umma_commit(&B.empty[slot]);
      }
      __syncwarp();
    };
    ok = mbar_wait_warp(&B.q_ready[t], i & 1u, abort);
    for (int v = 0; ok && v < C::kBufs && v < units; ++v) qk(v);
    for (int v = 0; ok && v < units; ++v) {
      const int k = tile_of(v), c = part_of(v);
      const uint32_t slot = slot_of(k, 1), u = u0 + (uint32_t)v, b = u % C::kBufs;
      if (split || !(v & 1)) ok = wait_tile(k, 1);
      ok = ok && mbar_wait_warp(&B.p_full[2 * t + b], (u / C::kBufs) & 1u, abort);
      if (!ok) break;
      tc_fence_after();
      const uint64_t dvs = dv + (uint64_t)((slot * C::kTBytes + c * 64 * 128) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int q = 0; q < kTerms; ++q)
#pragma unroll
          for (int s = 0; s < 4; ++s)
            umma_f16_ts(o_col, (q < 2 ? s_col + 64 * b + 32 * q : x_col + 32 * b) + 8 * s,
                        dvs + (uint64_t)((s * 2048) >> 4), C::kIdPV, q + s || v > 0 ? 1u : 0u);
        umma_commit(&B.pv_done[2 * t + b]);
        if (last_of(v)) umma_commit(&B.empty[slot]);
      }
      __syncwarp();
      if (v + C::kBufs < units) qk(v + C::kBufs);
    }
    // a tile of which this half had nothing (split, at most 64 tokens) is let go all the same
    if (ok && split && units < tiles)
      for (int part = 0; part < 2 && ok; ++part) {
        ok = wait_tile(tiles - 1, part);
        if (ok && elect_one()) umma_commit(&B.empty[slot_of(tiles - 1, part)]);
        __syncwarp();
      }
    if (elect_one()) umma_commit(&B.q_read[t]);  // the query operand may be replaced
    __syncwarp();
    tile0 += (uint32_t)tiles;
    u0 += (uint32_t)units;
  }
  drain_mmas(&B.drain[t]);
}

// ---------------------------------------------------------------- softmax (warps 0-7)

// A reference is rounded up, by as much as its last bit; up to this size the
// largest weight then keeps its place in f16 (bf16: in fp32's range).  A
// request whose reference passes it is refused.  (Rounding the scores as the
// reference was would resolve them, as the plain decode does, but a branch to
// that costs 2 to 9% of the kernel.)
template <bool kFp8>
constexpr float kMostRef = kFp8 ? 16777216.f : 536870912.f;  // 2^24, 2^29

template <bool kFp8, int kD, int kTerms, bool kToken>
__device__ __forceinline__ void softmax_rows(const PrefixArgs &a, uint8_t *smem, const PBars &B, uint32_t tmem,
                                             volatile int *abort) {
  using C = PCfg<kFp8, kD, kTerms>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = warp >> 2, r = (warp & 3) * 32 + lane;  // half, row of it
  const uint32_t tq = tmem + ((uint32_t)((warp & 3) * 32) << 16), col_o = tq + C::col_o(t);
  const int S = a.d.S;
  uint32_t tile0 = 0, u = 0;  // tiles before this item, this half's units so far
  for (uint32_t items = 0;; ++items) {
    if (!mbar_wait_warp(&B.item_full[items % kItemSlots], (items / kItemSlots) & 1u, abort)) return;
    const PItem it = reinterpret_cast<const PItem *>(smem + C::kOffItems)[items % kItemSlots];
    __syncwarp();
    if (lane == 0) mbar_arrive(&B.item_empty[items % kItemSlots]);
    if (it.n_rows == 0) return;
    const int n_tok = (it.p1 - it.p0) * S;
    const int row = it.split ? r : t * (kRows / 2) + r;  // row of the item's block
    const bool mine = row < it.n_rows;
    // this thread's query row into the operand; f16: scaled by 2^e, its largest value into [2^14, 2^15), exact down to
    // 2^-31 of that (smaller values are rounded to steps of 2^-24); the sign of the
    // factor that turns products into scores goes with it, so that the largest product is the largest score
    float mult = a.d.sm_scale_log2;
    if (kFp8 && !kToken) mult *= a.d.k_scale[it.h];
    // (the half's last QK^T of the item before has read the operand)
    if (items > 0 && !mbar_wait_warp(&B.q_read[t], (items - 1) & 1u, abort)) return;
    {
      uint4 x[kD / 8];
      const uint4 *src = nullptr;
      if (mine) {
        const int gr = it.row0 + row, b = a.members[it.first + gr / a.G];
        src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.d.q) +
                                              ((size_t)b * a.d.Hq + it.h * a.G + gr % a.G) * kD);
      }
#pragma unroll
      for (int j = 0; j < kD / 8; ++j) x[j] = mine ? src[j] : make_uint4(0u, 0u, 0u, 0u);
      float mx = 0.f;
#pragma unroll
      for (int j = 0; j < kD / 8; ++j) mx = amax8(x[j], mx);
      int e = 0;
      if (kFp8 && mx > 0.f) {
        frexpf(mx, &e);
        e = 15 - e;
      }
      // 2^e as two factors, either of which is a normal number
      float f1 = ldexpf(mult < 0.f ? -1.f : 1.f, e / 2);
      const float f2 = ldexpf(1.f, e - e / 2);
      mult = ldexpf(fabsf(mult), -e);
      if (mult == 0.f) {  // all scores are zero; a factor of zero would meet the masked tokens' -inf
        f1 = 0.f;
        mult = 1.f;
      }
      const uint32_t dst = smem_addr(smem + C::kOffQ) + t * C::kQBytes + r * 128;
#pragma unroll
      for (int j = 0; j < kD / 8; ++j) {
        uint32_t v[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float lo = __uint_as_float(v[q] << 16) * f1 * f2, hi = __uint_as_float(v[q] & 0xffff0000u) * f1 * f2;
          v[q] = kFp8 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
        }
        sts128(dst + (j >> 3) * C::kBlk + (((j & 7) ^ (r & 7)) << 4), make_uint4(v[0], v[1], v[2], v[3]));
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.q_ready[t]);
    }
    float m = kNegInf, l = 0.f, vref = 1.f;
    bool first = true;
    // 64 tokens of a tile at a time: both halves of it, or in split mode this half's
#pragma unroll 1
    for (int tok = it.split ? 64 * t : 0; tok < n_tok; tok += it.split ? kTok : 64) {
      const int valid = n_tok - tok;
      const uint32_t buf = u % C::kBufs, col = tq + C::col_s(t, 0) + 64 * buf, n = tile0 + (uint32_t)tok / kTok;
      const float *sc = reinterpret_cast<const float *>(smem + C::kOffScale) +
                        (n % C::kScaleSlots) * (2 * kTok + 4) + (tok & 64);
      if (!mbar_wait_warp(&B.s_full[2 * t + buf], (u / C::kBufs) & 1u, abort)) return;
      float moved = 1.f;
      if (kToken) {
        if (!mbar_wait_warp(&B.sc_full[n % C::kScaleSlots], (n / C::kScaleSlots) & 1u, abort)) return;
        const float now = sc[2 * kTok - (tok & 64)];  // against the reference this half last used
        if (!first && now != vref) moved = vref / now;
        vref = now;
      }
      tc_fence_after();
      uint32_t z[64];
      tmem_ld64(col, z);
      if (kToken) {
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
          const ulonglong2 k4 = *reinterpret_cast<const ulonglong2 *>(sc + j);
          const uint64_t s[2] = {k4.x, k4.y};
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float lo, hi;
            f32x2_split(mul_f32x2(f32x2(__uint_as_float(z[j + 2 * q]), __uint_as_float(z[j + 2 * q + 1])), s[q]), lo, hi);
            z[j + 2 * q] = __float_as_uint(lo);
            z[j + 2 * q + 1] = __float_as_uint(hi);
          }
        }
      }
      if (valid < 64) {
#pragma unroll
        for (int j = 0; j < 64; ++j)
          if (j >= valid) z[j] = 0xff800000u;
      }
      float part[2] = {kNegInf, kNegInf};
#pragma unroll
      for (int j = 0; j < 64; j += 2)  // three operands at a time
        part[j >> 1 & 1] = fmaxf(fmaxf(part[j >> 1 & 1], __uint_as_float(z[j])), __uint_as_float(z[j + 1]));
      float mx = fmaxf(part[0], part[1]);
      mx = mx == kNegInf ? kNegInf : __fmul_ru(mx, mult);  // no score is above it
      // move the reference
      const bool grow = mx - m > C::kGrow || first;
      if (__any_sync(0xffffffffu, grow || moved != 1.f)) {
        const float mn = grow ? __fsub_ru(mx, C::kLead) : m;
        const float al = first ? 0.f : fast_exp2(m - mn);
        l *= al;
        if (!first) {
          // after the products handed over last
          if (!mbar_wait_warp(&B.pv_done[2 * t + (u - 1) % C::kBufs], ((u - 1) / C::kBufs) & 1u, abort)) return;
          tc_fence_after();
          const float f = al * moved;
#pragma unroll 1
          for (int i = 0; i < kD / 32; ++i) {
            uint32_t o[32];
            tmem_ld32(col_o + 32 * i, o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st32(col_o + 32 * i, o);
          }
          tmem_wait_st();
        }
        m = mn;
      }
      first = false;
      const uint64_t mult2 = f32x2(mult, mult), off2 = f32x2(-m, -m);
      uint64_t sum = f32x2(0.f, 0.f);
      uint32_t pk[32];
#pragma unroll
      for (int k = 0; k < kTerms; ++k) {
#pragma unroll
        for (int j = 0; j < 64; j += 2) {
          uint64_t p = f32x2(__uint_as_float(z[j]), __uint_as_float(z[j + 1]));
          float p0, p1;
          if (k == 0) {
            f32x2_split(fma_f32x2(p, mult2, off2), p0, p1);
            p0 = fast_exp2(p0);
            p1 = fast_exp2(p1);
            p = f32x2(p0, p1);
            sum = add_f32x2(sum, p);
            if (kToken) p = mul_f32x2(p, reinterpret_cast<const uint64_t *>(sc + kTok)[j / 2]);
          }
          f32x2_split(p, p0, p1);
          pk[j / 2] = kFp8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
          if (k + 1 < kTerms) {  // what the next term carries
            float b0, b1;
            if constexpr (kFp8) {
              const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&pk[j / 2]));
              b0 = back.x;
              b1 = back.y;
            } else {
              b0 = __uint_as_float(pk[j / 2] << 16);
              b1 = __uint_as_float(pk[j / 2] & 0xffff0000u);
            }
            f32x2_split(fma_f32x2(f32x2(b0, b1), f32x2(-1.f, -1.f), p), p0, p1);
            z[j] = __float_as_uint(p0);
            z[j + 1] = __float_as_uint(p1);
          }
        }
        tmem_st32(k < 2 ? col + 32 * k : tq + C::col_x(t, 0) + 32 * buf, pk);
      }
      float sum0, sum1;
      f32x2_split(sum, sum0, sum1);
      l += sum0 + sum1;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.p_full[2 * t + buf]);
      ++u;
    }
    // the half's partial result
    if (!first) {
      if (!mbar_wait_warp(&B.pv_done[2 * t + (u - 1) % C::kBufs], ((u - 1) / C::kBufs) & 1u, abort)) return;
      tc_fence_after();
    }
    const float fac = !kFp8 ? 1.f : kToken ? vref : a.d.v_scale[it.h];
    const size_t at = (size_t)it.slot * kRows + t * (kRows / 2) + r;
#pragma unroll 1
    for (int i = 0; i < kD / 32; ++i) {
      uint32_t o[32];
      if (!first) {
        tmem_ld32(col_o + 32 * i, o);
      } else {  // split, and at most 64 tokens: half 1 has none
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = 0u;
      }
      if (mine)
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          float v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = __uint_as_float(o[j + q]) * fac;
          stg256(a.o + at * kD + 32 * i + j, v);
        }
    }
    if (mine) {
      a.ml[at] = make_float2(first ? kNegInf : m, l);
      // references only rise: none between was larger.  (Infinite ones give NaN, as in the plain decode.)
      if (!first && fabsf(m) >= kMostRef<kFp8> && fabsf(m) < INFINITY)
        atomicOr(&a.check_st[a.members[it.first + (it.row0 + row) / a.G]], PFKV_ST_RANGE);
    }
    tc_fence_before();
    tile0 += (uint32_t)(n_tok + kTok - 1) / kTok;
  }
}

template <bool kFp8, int kD, int kTerms, bool kToken>
__global__ void __launch_bounds__(kPThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                  const PrefixArgs a) {
  using C = PCfg<kFp8, kD, kTerms>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const PBars B = pbars_at(smem + C::kOffBars);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxSlots; ++i) {
      mbar_init(&B.full[i], kFp8 ? 4 : 1);
      mbar_init(&B.empty[i], 2);  // both halves
      mbar_init(&B.code_full[i], 1);
      mbar_init(&B.code_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.q_ready[i], 4);
      mbar_init(&B.q_read[i], 1);
      mbar_init(&B.drain[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&B.s_full[i], 1);
      mbar_init(&B.p_full[i], 4);
      mbar_init(&B.pv_done[i], 1);
    }
    for (int i = 0; i < kMaxSlots; ++i) mbar_init(&B.sc_full[i], 4);
    for (int i = 0; i < kItemSlots; ++i) {
      mbar_init(&B.item_full[i], 1);
      mbar_init(&B.item_empty[i], 10);  // eight softmax warps and the issuers
    }
    for (int i = 0; i < kTileSlots; ++i) {
      mbar_init(&B.tile_full[i], 1);
      mbar_init(&B.tile_empty[i], 4);
    }
    s_abort = 0;
    mbar_init_fence();
  }
  if (warp == 12) tmem_alloc(&s_tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)s_tmem);
  volatile int *abort = &s_abort;
  if (warp >= 12) regs_dec<kRegsRest>();
  if (warp == 13) {
    plan_tiles<kFp8, kD, kTerms, kToken>(a, map_k, map_v, smem, B, abort);
  } else {
    pdl_wait();
    pdl_launch_dependents();
    const PrefixHdr hdr = *a.hdr;
    if ((int)blockIdx.x < hdr.R) {
      if (warp < 8) {
        regs_inc<kRegsSoftmax>();
        softmax_rows<kFp8, kD, kTerms, kToken>(a, smem, B, tmem, abort);
      } else if (warp < 12) {
        regs_dec<kRegsLoader>();
        if constexpr (kFp8) loader_fp8<kFp8, kD, kTerms, kToken>(a, smem, B, abort);
      } else if (warp == 12) {
        issue_half<kFp8, kD, kTerms>(a, smem, B, tmem, 0, abort);
      } else if (warp == 14) {
        issue_half<kFp8, kD, kTerms>(a, smem, B, tmem, 1, abort);
      }
    }
    if (warp == 15) {
      find_pieces(a, hdr);
      check_prefixes(a, hdr);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0) a.aborts[blockIdx.x] = s_abort;
}

}  // namespace
}  // namespace pfkv
