"""A paged cache in plain Python: what the page operations do, one entry after
the other.  Everything is whole numbers and copies, so the GPU has to agree
exactly."""
import copy

import numpy as np


class Full(Exception):
    pass


class Bad(Exception):
    pass


class PageModel:
    def __init__(self, planes, pages, heads, ps, dim, seqs, max_pages, seed=0):
        self.ps, self.n_pages, self.max_pages, self.n_seqs = ps, pages, max_pages, seqs
        rng = np.random.default_rng(seed)
        self.pool = rng.integers(0, 2 ** 15, (planes, pages, heads, ps, dim)).astype(np.uint16) & 0x7BFF  # finite fp16
        self.ref = [0] * pages
        self.table = [[-1] * max_pages for _ in range(seqs)]
        self.len = [0] * seqs

    def _pages(self, n):
        return -(-n // self.ps)

    def _free(self, shared):
        return [p for p in range(self.n_pages) if shared[p] == 0]

    def _once(self, seqs):
        if len(set(seqs)) != len(seqs) or any(not 0 <= s < self.n_seqs for s in seqs):
            raise Bad

    def _all_or_nothing(self, f):
        keep = copy.deepcopy((self.pool, self.ref, self.table, self.len))
        try:
            f()
        except (Full, Bad):
            self.pool, self.ref, self.table, self.len = keep
            raise

    def fork(self, src, dst):
        def do():
            self._once(dst)
            if any(not 0 <= s < self.n_seqs or s in dst for s in src) or any(self.len[d] for d in dst):
                raise Bad
            for s, d in zip(src, dst):
                for i in range(self._pages(self.len[s])):
                    p = self.table[d][i] = self.table[s][i]
                    self.ref[p] += 1
                self.len[d] = self.len[s]
        self._all_or_nothing(do)

    def free(self, seqs):
        def do():
            self._once(seqs)
            for s in seqs:
                for i in range(self._pages(self.len[s])):
                    self.ref[self.table[s][i]] -= 1
                    self.table[s][i] = -1
                self.len[s] = 0
        self._all_or_nothing(do)

    def extend(self, seqs, add):
        def do():
            self._once(seqs)
            if any(a < 0 or self.len[s] + a > self.max_pages * self.ps for s, a in zip(seqs, add)):
                raise Bad
            shared = list(self.ref)
            free = self._free(shared)
            for s, a in zip(seqs, add):
                n = self.len[s]
                at = n // self.ps
                if a and n % self.ps and shared[self.table[s][at]] > 1:
                    if not free:
                        raise Full
                    old, new = self.table[s][at], free.pop(0)
                    self.pool[:, new, :, :n % self.ps] = self.pool[:, old, :, :n % self.ps]
                    self.ref[old] -= 1
                    self.ref[new] = 1
                    self.table[s][at] = new
                for i in range(self._pages(n), self._pages(n + a)):
                    if not free:
                        raise Full
                    self.table[s][i] = free.pop(0)
                    self.ref[self.table[s][i]] = 1
                self.len[s] = n + a
        self._all_or_nothing(do)

    def compact(self, seqs, base, keep):
        """keep[i]: a list, or None (left as it is)."""
        def do():
            self._once(seqs)
            for s, b, k in zip(seqs, base, keep):
                if k is None:
                    continue
                if not -1 <= b < self.len[s] or any(y <= x for x, y in zip([0] + k, k)) or (k and b + k[-1] >= self.len[s]):
                    raise Bad
            shared = list(self.ref)
            free = self._free(shared)
            before = self.pool.copy()
            for s, b, k in zip(seqs, base, keep):
                if k is None:
                    continue
                was, end = list(self.table[s]), b + 1 + len(k)
                d0 = next((d for d, x in enumerate(k) if x != d + 1), None)
                if d0 is not None:
                    first = b + 1 + d0
                    for i in range(first // self.ps, self._pages(end)):
                        if shared[was[i]] > 1:
                            if not free:
                                raise Full
                            self.table[s][i] = free.pop(0)
                            self.ref[was[i]] -= 1
                            self.ref[self.table[s][i]] = 1
                    for p in range(first // self.ps * self.ps, end):
                        src = p if p < first else b + k[p - b - 1]
                        self.pool[:, self.table[s][p // self.ps], :, p % self.ps] = before[:, was[src // self.ps], :, src % self.ps]
                for i in range(self._pages(end), self._pages(self.len[s])):
                    self.ref[self.table[s][i]] -= 1
                    self.table[s][i] = -1
                self.len[s] = end
        self._all_or_nothing(do)

    def copy(self, src, dst):
        for s, d in zip(src, dst):
            self.pool[:, d] = self.pool[:, s]

    def write(self, kp, vp, seqs, starts, k, v):
        for b, s in enumerate(seqs):
            m = starts[b + 1] - starts[b]
            for i in range(m):
                p = self.len[s] - m + i
                self.pool[kp, self.table[s][p // self.ps], :, p % self.ps] = k[starts[b] + i]
                self.pool[vp, self.table[s][p // self.ps], :, p % self.ps] = v[starts[b] + i]
