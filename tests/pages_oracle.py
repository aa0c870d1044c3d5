"""The pages of a cache by their definition, entry by entry on the host; no code of the
library. Contents of a block are one number (which contents it holds)."""
from __future__ import annotations

import numpy as np

BLOCK = 64


def blocks_of(tokens):
    return -(-int(tokens) // BLOCK)


class Pages:
    def __init__(self, slots, pool, width):
        self.table = np.full((slots, width), -1, np.int64)
        self.refs = np.zeros(pool, np.int64)
        self.held = np.arange(pool)      # contents of each block

    def _there(self, p):
        return 0 <= p < len(self.refs)

    def reserve(self, start, tokens):
        """Returns how many blocks are lacking."""
        entries = [(s, j) for s in range(len(self.table)) if start[s] >= 0 and tokens[s] > 0
                   for j in range(start[s] // BLOCK, min(blocks_of(int(start[s]) + int(tokens[s])), self.table.shape[1]))]
        writers = {}
        for e in entries:
            p = self.table[e]
            if self._there(p) and self.refs[p] > 1:
                writers.setdefault(p, []).append(e)
        need = []
        for e in entries:
            p = self.table[e]
            if not self._there(p):
                need.append(e)
            elif self.refs[p] > 1 and not (len(writers[p]) == self.refs[p] and writers[p][0] == e):
                need.append(e)
        free = [p for p in range(len(self.refs)) if self.refs[p] <= 0]
        if len(free) < len(need):
            return len(need) - len(free)
        for (s, j), q in zip(need, free):
            p = self.table[s, j]
            if self._there(p):
                if j * BLOCK < start[s]:
                    self.held[q] = self.held[p]
                self.refs[p] -= 1
            self.refs[q] = 1
            self.table[s, j] = q
        return 0

    def fork(self, source, length):
        old = self.table.copy()
        for s, f in enumerate(source):
            if 0 <= f < len(old):
                n = blocks_of(max(int(length[s]), 0))
                new = np.where(np.arange(old.shape[1]) < n, old[f], -1)
                for p in old[s]:
                    if self._there(p):
                        self.refs[p] -= 1
                for p in new:
                    if self._there(p):
                        self.refs[p] += 1
                self.table[s] = new

    def free(self, keep):
        for s, k in enumerate(keep):
            for j in range(blocks_of(max(int(k), 0)), self.table.shape[1]):
                if self._there(self.table[s, j]):
                    self.refs[self.table[s, j]] -= 1
                self.table[s, j] = -1

    def compact(self):
        """Returns the number of blocks in use and each block's place."""
        n = int((self.refs > 0).sum())
        moved = np.where(self.refs > 0, np.arange(len(self.refs)), -1)
        holes = [p for p in range(n) if self.refs[p] <= 0]
        for p, q in zip([p for p in range(n, len(self.refs)) if self.refs[p] > 0], holes):
            moved[p] = q
            self.held[q] = self.held[p]
            self.refs[q], self.refs[p] = self.refs[p], 0
        for e in np.ndindex(self.table.shape):
            p = self.table[e]
            if self._there(p) and moved[p] >= 0:
                self.table[e] = moved[p]
        return n, moved


def counts(table, pool):
    inside = table[(table >= 0) & (table < pool)]
    return np.bincount(inside, minlength=pool)
