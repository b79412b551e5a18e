// The work line of the shared-prefix decode, run on the host from the kernels'
// own functions (prefix.cuh): the pieces that the ranges write against those
// that the join looks for.
#include <map>

#include "prefix.cuh"

using namespace pfkv;

// Members and pages of each group, KV heads, query heads per KV head, page
// size, CTAs.  Returns how many (group, head, member, query head) rows do not
// find exactly the pages of their prefix, each once and in partial slots of
// their own row block; -1 where two pieces share a slot.
extern "C" long long prefix_line_faults(const int *members, const int *pages, int n_groups, int H, int G, int S,
                                        int ctas) {
  const LineUnits units = line_units(S);
  PrefixArgs a{};
  a.G = G;
  a.n_groups = n_groups;
  a.c0 = units.c0;
  a.d.cache.num_kv_heads = H;
  PrefixGroup groups[64];
  long long unit = 0;
  int first = 0, item = 0;
  for (int g = 0; g < n_groups; ++g) {
    const int p = members[g] ? pages[g] : 0;
    const HeadLine line = head_line(members[g], G, p, a.c0);
    groups[g] = PrefixGroup{first, members[g], first, 0, p, item, unit};
    first += members[g];
    item += p ? H * line.blocks : 0;
    unit += p ? H * line.head : 0;
  }
  const long long r = unit / units.min_units;
  const PrefixHdr hdr{unit, unit == 0 ? 0 : r < 1 ? 1 : (int)(r < ctas ? r : ctas), 0};
  std::map<long long, PItem> written;
  for (int k = 0; k < hdr.R; ++k) {
    PWalk w{range_start(hdr, k), range_start(hdr, k + 1), k};
    PItem it{};
    while (walk_next(a, groups, w, it))
      if (!written.emplace(it.slot, it).second) return -1;
  }
  long long faults = 0;
  for (int g = 0; g < n_groups; ++g)
    for (int rank = 0; groups[g].pages && rank < members[g]; ++rank)
      for (int hq = 0; hq < H * G; ++hq) {
        const PrefixRow pr = row_pieces(hdr, groups[g], G, a.c0, rank, hq);
        int at = 0;  // pages so far
        bool ok = true;
        for (int i = 0; i < pr.n >> pr.sh && ok; ++i) {
          const auto f = written.find(pr.slot0 + i);
          ok = f != written.end();
          if (!ok) break;
          const PItem &it = f->second;
          const int row = rank * G + hq % G - it.row0;
          ok = it.first == groups[g].first && it.h == hq / G && row == pr.row && row >= 0 && row < it.n_rows &&
               it.split == pr.sh && it.p0 == at && it.p1 > at;
          at = it.p1;
        }
        faults += !ok || at != groups[g].pages;
      }
  return faults;
}
