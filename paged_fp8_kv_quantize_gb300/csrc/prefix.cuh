// prefix.cuh -- decode attention of a batch that shares long prefixes: the
// plan, the work line and the workspace, shared by the kernels of
// prefix_attn.cu.
//
// The requests of a group g hold the same first p_g pages.  For KV head h the
// n_g G query rows of the group (n_g requests, G query heads each; row
// r = rank * G + j) are one matrix, which is cut into blocks of kRows rows;
// an item is one such block over the group's p_g pages.  The items, in order
// (group, KV head, block), lie on a line of
//   T = sum_g Hkv * ceil(n_g G / kRows) * p_g
// pages that is cut into R equal ranges, one per CTA; a piece is the part of
// one item inside one range.  The line's segments are numbered by the range
// and item boundaries before them, so piece (range k, item i) has partial slot
// k + i without a look at any other piece.
#pragma once

#include "decode_common.cuh"

namespace pfkv {
namespace {

constexpr int kMaxRanges = 256;  // CTAs of the prefix kernel at most
constexpr int kRows = 256;       // query rows of an item

struct PrefixGroup {
  int first, n;      // its requests: members[first .. first + n)
  int pages, item0;  // prefix pages, number of its first item
  long long unit0;   // its first page on the line
};

struct PrefixHdr {
  long long T;
  int R;  // ranges; 0 when no group has a prefix
  int pad;
};

struct PrefixArgs {
  DecodeArgs d;  // the decode call: cache, q, lengths, tables, workspace of the own pages' pieces, out, status
  int G;         // query heads per KV head
  const int *group_of, *group_pages;
  int n_groups;
  int ctas, min_pages;  // prefix kernel: CTAs, pages a range holds at least
  int out_bf16;
  // workspace
  int *own_len, *skip;  // [B] tokens past the prefix (0: none), prefix pages
  uint32_t *pre_st;     // [B] status bits of the plan
  int *rank, *members;  // [B] place of a request in its group; requests by group
  PrefixGroup *groups;  // [n_groups]
  PrefixHdr *hdr;
  float2 *ml;   // [slot][kRows]
  float *o;     // [slot][kRows][D]
  int *aborts;  // [kMaxRanges]
};

// floor(k T / R): first page of range k.
__device__ __forceinline__ long long range_start(const PrefixHdr &h, long long k) { return k * h.T / h.R; }
// The range that holds page u.
__device__ __forceinline__ int range_of(const PrefixHdr &h, long long u) { return (int)(((u + 1) * h.R - 1) / h.T); }

// Blocks of kRows rows that n requests' query rows of one KV head make.
__device__ __forceinline__ int row_blocks(int n, int G) { return (int)(((long long)n * G + kRows - 1) / kRows); }

}  // namespace
}  // namespace pfkv
