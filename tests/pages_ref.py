"""A plain model of the pages of a cache: one page and one sequence at a time (numpy, no library code)."""
import numpy as np


class Pool:
    def __init__(self, pages, page, sequences, width):
        self.page, self.width = page, width
        self.table = np.full((sequences, width), -1, np.int64)
        self.lens = np.zeros(sequences, np.int64)
        self.refs = np.zeros(pages, np.int64)
        self.left_out = 0

    def held(self, n):
        return -(-int(n) // self.page)

    def extend(self, cu, tokens):
        B = len(self.lens)
        slots, src, dst = np.full(tokens, -1, np.int64), np.full(B, -1, np.int64), np.full(B, -1, np.int64)
        free = list(np.flatnonzero(self.refs == 0))
        before = self.refs.copy()
        seen: dict = {}
        self.left_out, full = 0, False
        for b in range(B):
            a, z = int(cu[b]), int(cu[b + 1])
            if a == z:
                continue
            n, total = int(self.lens[b]), int(self.lens[b]) + z - a
            # positions that do not fit: the numbers of cu rise
            if not 0 <= a < z <= tokens or a < max(cu[:b + 1]) or total > self.width * self.page:
                self.left_out += 1
                continue
            copy = False
            if n % self.page:
                last = int(self.table[b, n // self.page])
                copy = before[last] - seen.get(last, 0) > 1
                seen[last] = seen.get(last, 0) + 1
            need = self.held(total) - self.held(n) + copy
            full = full or need > len(free)
            if full:
                self.left_out += 1
                continue
            if copy:
                src[b], dst[b] = last, free.pop(0)
                self.refs[last] -= 1
                self.refs[dst[b]] = 1
                self.table[b, n // self.page] = dst[b]
            for w in range(self.held(n), self.held(total)):
                self.table[b, w] = free.pop(0)
                self.refs[self.table[b, w]] = 1
            for t in range(a, z):
                at = n + t - a
                slots[t] = self.table[b, at // self.page] * self.page + at % self.page
            self.lens[b] = total
        return slots, src, dst

    def fork(self, parents):
        old, lens = self.table.copy(), self.lens.copy()
        for b, p in enumerate(parents):
            there = 0 <= p < len(lens)
            self.table[b] = old[p] if there else -1
            self.lens[b] = lens[p] if there else 0
        np.subtract.at(self.refs, old[old >= 0], 1)
        np.add.at(self.refs, self.table[self.table >= 0], 1)

    def truncate(self, lens):
        for b, n in enumerate(lens):
            if 0 <= n < self.lens[b]:
                for w in range(self.held(n), self.width):
                    if self.table[b, w] >= 0:
                        self.refs[self.table[b, w]] -= 1
                        self.table[b, w] = -1
                self.lens[b] = n

    def compact(self, most):
        src, dst = np.full(most, -1, np.int64), np.full(most, -1, np.int64)
        for i in range(most):
            free, live = np.flatnonzero(self.refs == 0), np.flatnonzero(self.refs)
            if not len(free) or not len(live) or free[0] > live[-1]:
                break
            src[i], dst[i] = live[-1], free[0]
            self.refs[dst[i]], self.refs[src[i]] = self.refs[src[i]], 0
            self.table[self.table == src[i]] = dst[i]
        return src, dst
