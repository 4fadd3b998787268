"""The paged KV cache, restated on lists and in float64 numpy.

``Pool`` follows the rules of ``q4_paged_reserve`` one request after another,
as they are worded: surplus pages return first, in order; then requests take
theirs from the end of the list, until the first for which it does not suffice.
"""
from collections import Counter

import numpy as np


class Pool:
    def __init__(self, slots, width, pages, page):
        self.width, self.pages, self.page = width, pages, page
        self.free = list(range(pages - 1, -1, -1))
        self.count = pages
        self.held = [0] * slots
        self.table = [[-1] * width for _ in range(slots)]

    def state(self):
        return np.array([self.count] + self.free + self.held + [x for r in self.table for x in r], dtype=np.int64)

    def reserve(self, offsets, slot, pos, total):
        """(slot_map, new_len, whether pages ran out, whether some request breaks a rule)."""
        S, page = len(slot), self.page
        slot_map, new_len = [-1] * total, [-1] * S
        if any(b < 0 or e < b or e > total for b, e in zip(offsets, offsets[1:])) or not 0 <= self.count <= self.pages:
            return slot_map, new_len, False, True
        need, good, times = [], [], Counter(slot)
        for s in range(S):
            rows = offsets[s + 1] - offsets[s]
            ok = 0 <= slot[s] < len(self.held) and times[slot[s]] == 1 and pos[s] >= 0 and \
                pos[s] + rows <= self.width * page
            ok = ok and 0 <= self.held[slot[s]] <= self.width and self.held[slot[s]] * page >= pos[s]
            need.append(-(-(pos[s] + rows) // page))
            good.append(ok)
        surplus = [(s, i) for s in range(S) if good[s] for i in range(need[s], self.held[slot[s]])]
        if self.count + len(surplus) > self.pages:
            return slot_map, new_len, False, True
        for s, i in surplus:
            self.free[self.count] = self.table[slot[s]][i]
            self.table[slot[s]][i] = -1
            self.count += 1
        wanted, top, short = 0, self.count, False
        for s in range(S):
            if not good[s]:
                continue
            have = self.held[slot[s]] = min(self.held[slot[s]], need[s])
            wanted += need[s] - have
            if need[s] > have and wanted > top:
                short = True
                continue
            for i in range(have, need[s]):
                self.count -= 1
                self.table[slot[s]][i] = self.free[self.count]
            self.held[slot[s]] = need[s]
            new_len[s] = pos[s] + offsets[s + 1] - offsets[s]
            for t in range(offsets[s], offsets[s + 1]):
                p = pos[s] + t - offsets[s]
                slot_map[t] = self.table[slot[s]][p // page] * page + p % page
        return slot_map, new_len, short, not all(good)


def rows_of(pages, ids, n):
    """Positions 0 .. n - 1 of a request, [n, heads, D], from pages [pages, heads, page, D] and its page numbers."""
    x = pages[np.asarray(ids)].transpose(0, 2, 1, 3)
    return x.reshape(-1, pages.shape[1], pages.shape[3])[:n]
