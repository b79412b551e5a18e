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
  int first, n;      // its requests: members[first .. first + n)
  int lead, pad;     // the first of them
  int pages, item0;  // prefix pages, number of its first item
  long long unit0;   // its first unit on the line
};

struct PrefixHdr {
  long long T;
  int R;  // ranges; 0 when no group has a prefix
  int pad;
};

// Where the join finds a row's pieces of the prefix: n of them, piece i in row
// `row` of slot0 + i, or, where an item's halves left one each (sh = 1), in row
// `row` + (i & 1) kRows / 2 of slot0 + i / 2.
struct PrefixRow {
  int slot0, n, row, sh;
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
  float2 *ml;   // [slot][kRows]
  float *o;     // [slot][kRows][D]
  int *aborts;  // [kMaxRanges]
};

// floor(k T / R): first unit of range k.
__device__ __forceinline__ long long range_start(const PrefixHdr &h, long long k) { return div_floor(k * h.T, h.R); }
// The range that holds unit u.
__device__ __forceinline__ int range_of(const PrefixHdr &h, long long u) {
  return (int)div_floor((u + 1) * h.R - 1, h.T);
}

// A group's items of one KV head on the line.
constexpr int kCostHalf = 4, kCostFull = 7;  // a page's cost; measured 1.2 and 2.1 us per 128 tokens (FP8, D 128)
struct HeadLine {
  int blocks, last_rows;       // row blocks, rows of the last one
  long long full, last, head;  // units of a full block, of the last one, of all
};
__device__ __forceinline__ HeadLine head_line(int n, int G, int pages, int c0) {
  HeadLine l;
  const long long rows = (long long)n * G;
  l.blocks = (int)((rows + kRows - 1) / kRows);
  l.last_rows = (int)(rows - (long long)(l.blocks - 1) * kRows);
  l.full = c0 + (long long)kCostFull * pages;
  l.last = c0 + (long long)(l.last_rows <= kRows / 2 ? kCostHalf : kCostFull) * pages;
  l.head = (l.blocks - 1) * l.full + l.last;
  return l;
}
__device__ __forceinline__ int page_cost(const HeadLine &l, int blk) {
  return blk == l.blocks - 1 && l.last_rows <= kRows / 2 ? kCostHalf : kCostFull;
}

}  // namespace
}  // namespace pfkv
