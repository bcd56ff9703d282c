"""A page table kept by plain sequential code, for comparison with the device's:
holders counted entry by entry, pages taken lowest id first, contents moved row
by row.  Shares nothing with the library."""

from __future__ import annotations

import numpy as np


def pages_of(tokens: int, page_size: int) -> int:
    return -(-tokens // page_size)


class PagesReference:
    def __init__(self, lens, table, num_pages, page_size, pools=()):
        self.lens = np.array(lens, np.int64)
        self.table = np.array(table, np.int64)
        self.N, self.P = num_pages, page_size
        self.pools = [np.array(p) for p in pools]
        self.ref = np.zeros(num_pages, np.int64)
        self.error = 0
        self.max_len = self.table.shape[1] * page_size
        for b, n in enumerate(self.lens):
            for p in range(pages_of(int(n), page_size)):
                self.ref[self.table[b, p]] += 1

    def flag(self, code):
        self.error = self.error or code

    def n_free(self):
        return int((self.ref == 0).sum())

    def fork(self, src, dst, tokens=None):
        start_lens = self.lens.copy()
        B = len(self.lens)
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < B and 0 <= d < B) or s == d or d in list(dst[:i]) \
                    or s in list(dst) or d in list(src) or start_lens[d] != 0:
                self.flag(7)
                continue
            n = int(start_lens[s]) if tokens is None or tokens[i] < 0 else int(tokens[i])
            if n > start_lens[s]:
                self.flag(3)
                continue
            for p in range(pages_of(n, self.P)):
                self.table[d, p] = self.table[s, p]
                self.ref[self.table[s, p]] += 1
            self.lens[d] = n

    def free(self, rows, keep=None):
        seen = set()
        for i, r in enumerate(rows):
            k = 0 if keep is None else int(keep[i])
            if not 0 <= r < len(self.lens) or r in seen:
                self.flag(7)
                continue
            seen.add(r)
            if not 0 <= k <= self.lens[r]:
                self.flag(3)
                continue
            for p in range(pages_of(k, self.P), pages_of(int(self.lens[r]), self.P)):
                self.ref[self.table[r, p]] -= 1
                self.table[r, p] = -1
            self.lens[r] = k

    def extend(self, add):
        B = len(self.lens)
        if any(a < 0 or n + a > self.max_len for n, a in zip(self.lens, add)):
            self.flag(3)
            return False
        grows = {}  # shared partial page -> its growing rows
        for b in range(B):
            if add[b] > 0 and self.lens[b] % self.P:
                grows.setdefault(int(self.table[b, self.lens[b] // self.P]), []).append(b)
        copies = set()
        for page, rows in grows.items():
            stay = rows[-1:] if len(rows) == self.ref[page] else []
            copies |= {r for r in rows if r not in stay and self.ref[page] > 1}
        need = [int(add[b] > 0) * (pages_of(int(self.lens[b] + add[b]), self.P)
                                   - pages_of(int(self.lens[b]), self.P)) + (b in copies)
                for b in range(B)]
        free = [int(p) for p in np.nonzero(self.ref == 0)[0]]
        if sum(need) > len(free):
            self.flag(6)
            return False
        for b in range(B):
            n, a = int(self.lens[b]), int(add[b])
            if b in copies:
                old, new = int(self.table[b, n // self.P]), free.pop(0)
                for pool in self.pools:
                    pool[new, : n % self.P] = pool[old, : n % self.P]
                self.ref[old] -= 1
                self.ref[new] = 1
                self.table[b, n // self.P] = new
            for p in range(pages_of(n, self.P), pages_of(n + a, self.P)):
                new = free.pop(0)
                self.table[b, p] = new
                self.ref[new] = 1
            self.lens[b] = n + a
        return True

    def compact(self):
        used = np.nonzero(self.ref)[0]
        n_used = len(used)
        page_map = np.full(self.N, -1, np.int64)
        page_map[used] = used
        high = [p for p in used if p >= n_used]
        holes = [p for p in range(n_used) if self.ref[p] == 0]
        for s, d in zip(high, holes):
            page_map[s] = d
            for pool in self.pools:
                pool[d] = pool[s]
            self.ref[d], self.ref[s] = self.ref[s], 0
        for b, n in enumerate(self.lens):
            for p in range(pages_of(int(n), self.P)):
                self.table[b, p] = page_map[self.table[b, p]]
        return page_map
