// prefix.cuh -- decode attention of a batch that shares long prefixes: the
// plan, the work line and the workspace, shared by the kernels of
// prefix_attn.cu.
//
// The requests of a group g hold the same first p_g pages.  For KV head h the
// n_g G query rows of the group (n_g requests, G query heads each; row
// r = rank * G + j) are one matrix, which is cut into blocks of kRows rows;
// an item is one such block over the group's p_g pages.  The items, in order
// (group, KV head, block), lie on a line of cost units: c0 for an item's
// set-up and read-out, then kCostFull a page (kCostHalf in a block of at most
// kRows / 2 rows).  The line, T units long, is cut into R equal ranges, one per
// CTA; a piece is the pages of one item that begin inside one range.  The
// line's segments are numbered by the range and item boundaries before them,
// so piece (range k, item i) has partial slot k + i without a look at any other
// piece.
#pragma once

#include "decode_common.cuh"

namespace pfkv {
namespace {

constexpr int kMaxRanges = 256;  // CTAs of the prefix kernel at most
constexpr int kRows = 256;       // query rows of an item

struct PrefixGroup {
  int first, n;      // its requests: members[first .. first + n), those whose length covers the prefix
  int lead, pad;     // the first of them
  int pages, item0;  // prefix pages, number of its first item
  long long unit0;   // its first unit on the line
};

struct PrefixHdr {
  long long T;
  int R;          // ranges; 0 when no group has a prefix
  int max_pages;  // pages of the longest prefix
};

// Where the join finds a row's pieces of the prefix: n of them, piece i in row
// `row` of slot0 + i, or, where an item's halves left one each (sh = 1), in row
// `row` + (i & 1) kRows / 2 of slot0 + i / 2.
struct PrefixRow {
  int slot0, n, row, sh;
};

// One piece of work; n_rows 0 ends the work.
struct PItem {
  int first, lead, row0, n_rows, h, p0, p1;
  long long slot;
  int split;  // at most 128 rows: each half takes 64 tokens of a tile
};
static_assert(sizeof(PItem) % 8 == 0, "tile slots follow it in shared memory");

// A range's first piece, and where the walk goes on from there.
struct PRange {
  PItem item;
  long long u, u1;
};

struct PrefixArgs {
  DecodeArgs d;  // the decode call: cache, q, lengths, tables, workspace of the own pages' pieces, out, status
  int G;         // query heads per KV head
  const int *group_of, *group_pages;
  int n_groups;
  int ctas;       // CTAs of the prefix kernel
  int c0;         // units of an item's set-up and read-out
  int min_units;  // units a range holds at least
  int out_bf16;
  // workspace
  int *own_len, *skip;  // [B] tokens past the prefix (0: none), prefix pages
  uint32_t *pre_st;     // [B] status bits of the plan
  uint32_t *check_st;   // [B] status bits of the prefix pages
  int *rank, *members;  // [B] place of a request in its group; requests by group
  PrefixGroup *groups;  // [n_groups]
  PrefixRow *rows;      // [B][Hq], written beside the products
  PrefixHdr *hdr;
  PRange *ranges;  // [kMaxRanges]
  float2 *ml;   // [slot][kRows]
  float *o;     // [slot][kRows][D]
  int *aborts;  // [kMaxRanges]
};

// floor(k T / R): first unit of range k.
__host__ __device__ __forceinline__ long long range_start(const PrefixHdr &h, long long k) {
  return div_floor(k * h.T, h.R);
}
// The range that holds unit u.
__host__ __device__ __forceinline__ int range_of(const PrefixHdr &h, long long u) {
  return (int)div_floor((u + 1) * h.R - 1, h.T);
}

// A page's cost: about 1.1 us and 1.8 us per 128 tokens for FP8 caches of head
// dimension 128, and used for all.  (They only weigh blocks of at most half the
// rows against the others, on a line that has both.)
constexpr int kCostHalf = 4, kCostFull = 7;

// Units of an item's set-up and read-out, about what 512 tokens of a small
// block cost, and units that a range holds at least: 256 such tokens, and one
// page of any block.  With less than a page a range between an item's first
// and last one may hold no page's beginning; nobody then writes the slot that
// row_pieces counts there.
struct LineUnits {
  int c0, min_units;
};
inline LineUnits line_units(int S) {
  const int units = kCostHalf * ((256 + S - 1) / S);
  return {kCostHalf * ((512 + S - 1) / S), units > kCostFull ? units : kCostFull};
}

// A group's items of one KV head on the line.
struct HeadLine {
  int blocks, last_rows;       // row blocks, rows of the last one
  long long full, last, head;  // units of a full block, of the last one, of all
};
__host__ __device__ __forceinline__ HeadLine head_line(int n, int G, int pages, int c0) {
  HeadLine l;
  const long long rows = (long long)n * G;
  l.blocks = (int)((rows + kRows - 1) / kRows);
  l.last_rows = (int)(rows - (long long)(l.blocks - 1) * kRows);
  l.full = c0 + (long long)kCostFull * pages;
  l.last = c0 + (long long)(l.last_rows <= kRows / 2 ? kCostHalf : kCostFull) * pages;
  l.head = (l.blocks - 1) * l.full + l.last;
  return l;
}
__host__ __device__ __forceinline__ int page_cost(const HeadLine &l, int blk) {
  return blk == l.blocks - 1 && l.last_rows <= kRows / 2 ? kCostHalf : kCostFull;
}
// Pages of that cost that begin before unit x of an item's pages.
__host__ __device__ __forceinline__ int pages_before(long long x, int cost) {
  if (x <= 0) return 0;
  const unsigned long long y = (unsigned long long)x + (unsigned)(cost - 1);
  return (int)(cost == kCostHalf ? y / kCostHalf : y / kCostFull);
}

// The pieces of query head hq's row of the rank-th request of a group.
__host__ __device__ __forceinline__ PrefixRow row_pieces(const PrefixHdr &hdr, const PrefixGroup &gr, int G, int c0,
                                                         int rank, int hq) {
  const HeadLine line = head_line(gr.n, G, gr.pages, c0);
  const int h = hq / G, r = rank * G + hq % G, blk = r / kRows;
  const int item = h * line.blocks + blk, cost = page_cost(line, blk);
  const long long first = gr.unit0 + h * line.head + blk * line.full + c0;  // unit of its first page
  const int k0 = range_of(hdr, first);
  PrefixRow pr;
  pr.sh = cost == kCostHalf;
  pr.n = (range_of(hdr, first + (long long)cost * (gr.pages - 1)) - k0 + 1) << pr.sh;
  pr.slot0 = k0 + gr.item0 + item;
  pr.row = r - blk * kRows;
  return pr;
}

// The pieces of range k from unit u on.
struct PWalk {
  long long u, u1;
  int k;
};

// The next piece with pages.
__host__ __device__ __forceinline__ bool walk_next(const PrefixArgs &a, const PrefixGroup *groups, PWalk &w, PItem &it) {
  while (w.u < w.u1) {
    int lo = 0, hi = a.n_groups - 1;  // the last group that starts at or before u
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (groups[mid].unit0 <= w.u) lo = mid;
      else hi = mid - 1;
    }
    const PrefixGroup g = groups[lo];
    const HeadLine line = head_line(g.n, a.G, g.pages, a.c0);
    const long long rel = w.u - g.unit0;
    it.h = (int)div_floor(rel, line.head);
    const long long in_head = rel - it.h * line.head;
    const int blk = line.blocks == 1 ? 0 : (int)min((long long)(line.blocks - 1), div_floor(in_head, line.full));
    const long long off = in_head - blk * line.full, seg = blk < line.blocks - 1 ? line.full : line.last;
    const long long end = min(seg, off + (w.u1 - w.u));
    const int cost = page_cost(line, blk);
    it.p0 = pages_before(off - a.c0, cost);
    it.p1 = pages_before(end - a.c0, cost);
    w.u += end - off;
    if (it.p1 <= it.p0) continue;
    it.first = g.first;
    it.lead = g.lead;
    it.row0 = blk * kRows;
    it.n_rows = blk < line.blocks - 1 ? kRows : line.last_rows;
    it.slot = (long long)w.k + g.item0 + it.h * line.blocks + blk;
    it.split = cost == kCostHalf;
    return true;
  }
  return false;
}

}  // namespace
}  // namespace pfkv
