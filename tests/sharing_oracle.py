"""Sequential reference of the page operators (copy, fork, release, compact):
plain Python over numpy arrays, one entry after another, as the header
describes them.  Test infrastructure only."""
from __future__ import annotations

from collections import Counter

import numpy as np

STALE_TAG, PAGE_OOB, BAD_LEN, NO_PAGES, NOT_HELD, DUPLICATE, BAD_ROW = 1, 2, 4, 16, 32, 64, 128


class SharedPool:
    """A pool of P pages: free stack (last one handed out first), held flags,
    tags, holder counts, and any number of per-page arrays [P][H][S][...]."""

    def __init__(self, P, page_tags, arrays):
        self.P = P
        self.tags = page_tags.copy()
        self.held = np.zeros(P, dtype=bool)
        self.refs = np.zeros(P, dtype=np.int32)
        self.stack = list(range(P - 1, -1, -1))
        self.arrays = [a.copy() for a in arrays]
        self.S = arrays[0].shape[2]

    def take(self):
        p = self.stack.pop()
        self.held[p] = True
        self.tags[p] = (int(self.tags[p]) + 1) & 0xFFFFFFFF
        return p

    def alloc(self, n):
        return [self.take() for _ in range(n)] if n <= len(self.stack) else None

    def copy(self, src, dst, slots=None):
        st = np.zeros(len(src), dtype=np.uint32)
        for i, (s, d) in enumerate(zip(src, dst)):
            n = self.S if slots is None else int(slots[i])
            if not (0 <= s < self.P and 0 <= d < self.P):
                st[i] |= PAGE_OOB
            if not 0 <= n <= self.S:
                st[i] |= BAD_LEN
            if st[i] == 0:
                for a in self.arrays:
                    a[d][:, :n] = a[s][:, :n]
        return st

    def fork(self, parents, children, lens, table, btags, tag_check):
        n, (B, MP), S = len(parents), table.shape, self.S
        st = np.zeros(n, dtype=np.uint32)
        for i in range(n):
            par, chi, m = int(parents[i]), int(children[i]), int(lens[i])
            if not (0 <= par < B and 0 <= chi < B):
                st[i] |= BAD_ROW
            if not 0 <= m <= MP * S:
                st[i] |= BAD_LEN
            if chi in children[:i] or chi in parents:
                st[i] |= DUPLICATE
            if st[i] & (BAD_ROW | BAD_LEN):
                continue
            for k in range(-(-m // S)):
                p = int(table[par, k])
                if not 0 <= p < self.P:
                    st[i] |= PAGE_OOB
                    continue
                if not self.held[p]:
                    st[i] |= NOT_HELD
                if tag_check and self.tags[p] != btags[par, k]:
                    st[i] |= STALE_TAG
        sound = [i for i in range(n) if st[i] == 0]
        if sum(int(lens[i]) % S != 0 for i in sound) > len(self.stack):
            st[sound] = NO_PAGES
            return st
        for i in sound:
            par, chi, m = int(parents[i]), int(children[i]), int(lens[i])
            full, tail = divmod(m, S)
            for k in range(full):
                table[chi, k], btags[chi, k] = table[par, k], btags[par, k]
                self.refs[table[par, k]] += 1
            if tail:
                p = self.take()
                table[chi, full], btags[chi, full] = p, self.tags[p]
                for a in self.arrays:
                    a[p][:, :tail] = a[table[par, full]][:, :tail]
        return st

    def release(self, pages):
        st = np.zeros(len(pages), dtype=np.uint32)
        ids = [int(p) for p in pages]
        over = {p for p, n in Counter(ids).items() if 0 <= p < self.P and n > self.refs[p] + 1}
        for i, p in enumerate(ids):
            if not 0 <= p < self.P:
                st[i] = PAGE_OOB
            elif not self.held[p]:
                st[i] = NOT_HELD
            elif self.refs[p] > 0 and p not in over:
                self.refs[p] -= 1
            else:  # the last holder, or more listings than holders
                self.refs[p] = 0
                self.held[p] = False
                self.stack.append(p)
        return st

    def compact(self, table, btags, used, max_moves):
        n_live = np.full(table.shape[0], table.shape[1]) if used is None else np.asarray(used)
        live = np.arange(table.shape[1]) < n_live[:, None]
        moves = []
        while len(moves) < max_moves:
            h, f = np.flatnonzero(self.held), np.flatnonzero(~self.held)
            if not h.size or not f.size or h[-1] < f[0]:
                break
            s, d = int(h[-1]), int(f[0])
            self.held[s], self.held[d] = False, True
            self.refs[d], self.refs[s] = self.refs[s], 0
            self.tags[d] = (int(self.tags[d]) + 1) & 0xFFFFFFFF
            for a in self.arrays:
                a[d] = a[s]
            named = live & (table == s)
            if btags is not None:
                named &= btags == self.tags[s]
                btags[named] = self.tags[d]
            table[named] = -2 - d  # not a page of a later move
            moves.append((s, d))
        table[table <= -2] = -2 - table[table <= -2]
        self.stack = sorted(np.flatnonzero(~self.held).tolist(), reverse=True)
        return moves
