"""Plain forms of a beam search's step and of the calls that keep a paged cache's pages, written
from the definitions in the header, one thing at a time; and states to run them on."""
import math

import numpy as np


# ------------------------------------------------------------------ beam selection

def select(x, scores, lengths, end, alpha, ended):
    """x [B, K, V] in 64 bits; ended: (scores, rows, lengths) [B, K]. Returns tokens, parents, scores,
    the new `ended`, and the sentences whose candidates are told apart by less than 1e-6 (what
    32-bit sums may turn round)."""
    B, K, V = x.shape
    tokens, parents = np.zeros((B, K), np.int32), np.zeros((B, K), np.int32)
    out, close = np.full((B, K), -np.inf), []
    ended = [np.array(a) for a in ended]
    for b in range(B):
        pairs = []
        for k in range(K):
            s, row = float(scores[b, k]), x[b, k]
            if s == -np.inf or not s < np.inf or np.isnan(row).any() or row.max() in (np.inf, -np.inf):
                continue
            top = row.max()
            total = s - math.log(np.exp(row - top).sum()) + (row - top)
            best = np.argsort(-total, kind="stable")[:2 * K + 1]
            pairs += [(-total[v], k * V + v) for v in best if total[v] > -np.inf]
        pairs.sort()
        n = 2 * K if end >= 0 else K
        near = pairs[:n + 1]
        if any(q[0] - p[0] < 1e-6 and p[1] // V != q[1] // V for p, q in zip(near, near[1:])):
            close.append(b)
        goes = [p for p in pairs[:n] if p[1] % V != end]
        for k in range(K):
            if k < len(goes):
                out[b, k], tokens[b, k], parents[b, k] = -goes[k][0], goes[k][1] % V, b * K + goes[k][1] // V
            else:
                tokens[b, k], parents[b, k] = max(end, 0), b * K + k
        if end >= 0:
            length = max(int(lengths[b]), 1)
            old = [(float(ended[0][b, k]), int(ended[1][b, k]), int(ended[2][b, k])) for k in range(K)]
            old = [o for o in old if o[0] > -np.inf]
            old += [(float(np.float32(-t / ((5 + length) / 6) ** alpha)), b * K + at // V, length)
                    for t, at in pairs[:n] if at % V == end]
            old.sort(key=lambda o: -o[0])
            ended[0][b] = -np.inf
            for k, o in enumerate(old[:K]):
                ended[0][b, k], ended[1][b, k], ended[2][b, k] = o
    return tokens, parents, out, ended, close


# ------------------------------------------------------------------ pages

class Pages:
    """A table and its counts as lists, changed an entry at a time."""

    def __init__(self, table, counts, page_size):
        self.table, self.counts, self.page = [list(map(int, r)) for r in table], list(map(int, counts)), page_size

    def put(self, b, k, page):
        old = self.table[b][k]
        if 0 <= old < len(self.counts):
            self.counts[old] -= 1
        self.table[b][k] = page
        if 0 <= page < len(self.counts):
            self.counts[page] += 1

    def fork(self, parents):
        old = [list(r) for r in self.table]
        for b, parent in enumerate(parents):
            if parent == b or parent < -1 or parent >= len(old):
                continue
            for k in range(len(old[b])):
                self.put(b, k, old[parent][k] if parent >= 0 else -1)

    def release(self, keep):
        for b, n in enumerate(keep):
            if n >= 0:
                for k in range(-(-int(n) // self.page), len(self.table[b])):
                    self.put(b, k, -1)

    def reserve(self, lens, new):
        """Returns (copies, missing)."""
        wanted, writers = [], {}
        for b, (n, m) in enumerate(zip(lens, new)):
            start, end = max(n - m, 0), min(n, len(self.table[b]) * self.page)
            if m > 0 and end > start:
                wanted += [(b, k, start - k * self.page) for k in range(start // self.page, -(-end // self.page))]
        for b, k, _ in wanted:
            p = self.table[b][k]
            if 0 <= p < len(self.counts):
                writers.setdefault(p, []).append(b)
        moves = []
        for b, k, rows in wanted:
            p = self.table[b][k]
            if not 0 <= p < len(self.counts):
                moves.append((b, k, -1, 0))
            elif self.counts[p] > 1 and not (len(writers[p]) == self.counts[p] and min(writers[p]) == b):
                moves.append((b, k, p, max(rows, 0)))
        free = [p for p, c in enumerate(self.counts) if c == 0]
        if len(moves) > len(free):
            return [], len(moves) - len(free)
        copies = []
        for (b, k, p, rows), to in zip(moves, free):
            if rows:
                copies.append((p, to, rows))
            self.put(b, k, to)
        return copies, 0

    def compact(self, max_copies):
        """Returns (copies, used)."""
        used = sum(c != 0 for c in self.counts)
        holes = [p for p in range(used) if self.counts[p] == 0]
        movers = [p for p in range(len(self.counts) - 1, used - 1, -1) if self.counts[p] != 0]
        copies = list(zip(movers, holes))[:max_copies]
        for src, dst in copies:
            self.counts[dst], self.counts[src] = self.counts[src], 0
        to = dict(copies)
        self.table = [[to.get(p, p) for p in r] for r in self.table]
        return [(s, d, self.page) for s, d in copies], used


def state(rng, B, max_pages, n_pages, page_size, share=0.3, held=None):
    """A table [B, max_pages] whose rows hold some pages, part of them shared with the row before,
    over a pool of n_pages in random order, and its counts."""
    order = list(rng.permutation(n_pages))
    table = np.full((B, max_pages), -1, np.int32)
    for b in range(B):
        n = int(rng.integers(0, max_pages + 1)) if held is None else held[b]
        shared = 0
        if b and rng.random() < 0.7:
            before = int((table[b - 1] >= 0).sum())
            shared = min(n, before, int(rng.integers(0, max_pages + 1) if rng.random() < share * 2 else 0))
            table[b, :shared] = table[b - 1, :shared]
        for k in range(shared, n):
            if order:
                table[b, k] = order.pop()
    counts = np.bincount(table[table >= 0], minlength=n_pages).astype(np.int32)
    return table, counts
