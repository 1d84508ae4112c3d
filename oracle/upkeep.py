"""What the pool's books and the acceptance of drafts do, written from their definitions: the
books as plain lists changed one sequence after the other, acceptance in whole numbers of any
length. No tensor arithmetic and none of the library's code."""
from __future__ import annotations

from fractions import Fraction

BOUNDS, FULL, VALUE = 2, 8, 16          # flags: lengths (1: block ids), too few free blocks, values


class Books:
    """The books of a pool; every call returns (flags, copies, blocks left), flags 0 if it was done."""

    def __init__(self, max_seqs, max_blocks, num_blocks, block_size):
        self.W, self.bs = max_blocks, block_size
        self.rows = [[] for _ in range(max_seqs)]
        self.lens = [0] * max_seqs
        self.ref = [0] * num_blocks

    @classmethod
    def of(cls, table, lens, ref, block_size):
        k = cls(len(lens), len(table[0]), len(ref), block_size)
        k.lens, k.ref = list(lens), list(ref)
        k.rows = [list(r[:-(-n // block_size)]) for r, n in zip(table, lens)]
        return k

    def table(self):
        return [r + [-1] * (self.W - len(r)) for r in self.rows]

    def free(self):
        return [i for i, c in enumerate(self.ref) if c == 0]

    def _longest(self):
        return min(self.W * self.bs, 2 ** 31 - 256)

    def resize(self, new):
        free, copies, before = self.free(), [], list(self.ref)
        if any(not 0 <= n <= self._longest() for n in new):
            return BOUNDS, [], len(free)
        blocks = [-(-n // self.bs) for n in new]
        split = [n < l and n % self.bs and before[r[k - 1]] > 1 for n, l, r, k in zip(new, self.lens, self.rows, blocks)]
        if sum(max(0, k - len(r)) + bool(x) for k, r, x in zip(blocks, self.rows, split)) > len(free):
            return FULL, [], len(free)
        for b, (n, k) in enumerate(zip(new, blocks)):
            row = self.rows[b]
            if split[b]:
                old, row[k - 1] = row[k - 1], free.pop(0)
                self.ref[old] -= 1
                self.ref[row[k - 1]] = 1
                copies.append([old, row[k - 1], 0, n % self.bs])
            while len(row) < k:
                row.append(free.pop(0))
                self.ref[row[-1]] = 1
            while len(row) > k:
                self.ref[row.pop()] -= 1
            self.lens[b] = n
        return 0, copies, self.ref.count(0)

    def fork(self, parents, children, lens=None):
        free, copies, S = self.free(), [], len(self.lens)
        if any(not (0 <= a < S and 0 <= c < S) for a, c in zip(parents, children)) or len(set(children)) < len(children):
            return BOUNDS, [], len(free)
        lens = [self.lens[a] for a in parents] if lens is None else lens
        if any(not 0 <= n <= self.lens[a] or self.lens[c] for a, c, n in zip(parents, children, lens)):
            return BOUNDS, [], len(free)
        if sum(n % self.bs > 0 for n in lens) > len(free):
            return FULL, [], len(free)
        for a, c, n in zip(parents, children, lens):
            row = self.rows[a][:n // self.bs]
            for i in row:
                self.ref[i] += 1
            if n % self.bs:
                row.append(free.pop(0))
                self.ref[row[-1]] = 1
                copies.append([self.rows[a][n // self.bs], row[-1], 0, n % self.bs])
            self.rows[c], self.lens[c] = row, n
        return 0, copies, self.ref.count(0)

    def compact(self, room):
        live = sum(c > 0 for c in self.ref)
        high = [i for i in range(live, len(self.ref)) if self.ref[i]]
        holes = [i for i in range(live) if not self.ref[i]]
        pairs = list(zip(high, holes))[:room]
        to = dict(pairs)
        for a, b in pairs:
            self.ref[b], self.ref[a] = self.ref[a], 0
        self.rows = [[to.get(i, i) for i in r] for r in self.rows]
        return 0, [[a, b, 0, self.bs] for a, b in pairs], live


def accept(p, q, x, u, counts=None, lens=None):
    """p [B][K + 1][V], q [B][K][V] or None, x [B][K], u [B][K + 1] (floats) -> per sequence
    (flags, accepted, tokens, new length)."""
    out = []
    for b in range(len(p)):
        K, V = len(p[b]) - 1, len(p[b][0])
        k = K if counts is None else counts[b]
        n0 = 0 if lens is None else lens[b]
        if k < 0:
            out.append((0, 0, [-1] * (K + 1), n0))
            continue
        if lens is not None and n0 < K:
            out.append((BOUNDS, 0, [-1] * (K + 1), n0))
            continue
        nothing = (VALUE, 0, [-1] * (K + 1), n0 - K)
        if k > K or not 0 <= u[b][K] <= 1 or any(not 0 <= i < V for i in x[b][:k]):
            out.append(nothing)
            continue
        read = [p[b][i][x[b][i]] for i in range(k)] + [u[b][i] for i in range(k)]
        read += [q[b][i][x[b][i]] for i in range(k)] if q is not None else []
        if any(not 0 <= v <= 1 for v in read):
            out.append(nothing)
            continue
        n = 0
        while n < k and Fraction(u[b][n]) * (1 if q is None else Fraction(q[b][n][x[b][n]])) < Fraction(p[b][n][x[b][n]]):
            n += 1
        row = p[b][n]
        if any(not 0 <= v <= 1 for v in row) or (n < k and q is not None and any(not 0 <= v <= 1 for v in q[b][n])) or sum(row) > 2:
            out.append(nothing)
            continue
        whole = [round(v * 2.0 ** 46) for v in row]
        w = whole
        if n < k:
            less = [2 ** 46 * (j == x[b][n]) for j in range(V)] if q is None else [round(v * 2.0 ** 46) for v in q[b][n]]
            w = [max(i - j, 0) for i, j in zip(whole, less)]
            w = w if any(w) else whole
        total = sum(w)
        if not total:
            out.append(nothing)
            continue
        border, at, token = Fraction(u[b][K]) * total, 0, None
        for j, v in enumerate(w):
            at += v
            if v and (token is None or u[b][K] == 1):
                token = j if at > border or u[b][K] == 1 else None
        out.append((0, n, list(x[b][:n]) + [token] + [-1] * (K - n), n0 - K + n))
    return out
