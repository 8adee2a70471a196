"""The 4-bit cache format and the page operations in numpy, from their
definitions (64-bit arithmetic, Python loops over pages); not collected."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# e4m3: 4 exponent bits (bias 7), 3 mantissa bits, 0x7F is NaN
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:-1])
HALF, PAGE = 1152, 16


def nearest(x, grid):
    """Index of the grid value nearest to each x >= 0 (ascending grid, saturating, ties to the even index)."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    down, up = x - grid[lo], grid[hi] - x
    return np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def encode(x, g):
    """Rows [..., 128] -> (codes [..., 64] uint8, scales [..., 8] uint8)."""
    x = np.asarray(x, np.float64).reshape(*x.shape[:-1], 8, 16) / g
    si = nearest(np.abs(x).max(-1) / 6, E4M3)
    s = E4M3[si][..., None]
    ci = np.where(s > 0, nearest(np.abs(x) / np.where(s > 0, s, 1), E2M1), 0) + 8 * (x < 0)
    ci = ci.reshape(*x.shape[:-2], 128).astype(np.uint8)
    return ci[..., 0::2] | ci[..., 1::2] << 4, si.astype(np.uint8)


def decode(codes, scales, g):
    ci = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 8, 16)
    sign = np.where(ci >= 8, -1.0, 1.0)
    s = np.append(E4M3, np.nan)[scales & 127] * np.where(scales >= 128, -1.0, 1.0)
    return (sign * E2M1[ci & 7] * s[..., None] * g).reshape(*codes.shape[:-1], 128)


def put(pool, table, b, pos, which, rows, g):
    """Rows [m, hkv, 128] to positions pos .. pos + m - 1 of sequence b of a numpy pool."""
    for i, row in enumerate(rows):
        page, tok = table[b, (pos + i) // PAGE], (pos + i) % PAGE
        codes, scales = encode(row, g)
        pool[page, :, which, tok * 64:tok * 64 + 64] = codes
        pool[page, :, which, 1024 + tok * 8:1024 + tok * 8 + 8] = scales


def get(pool, table, b, pos, m, which, g):
    """[m, hkv, 128] float64 of positions pos .. pos + m - 1."""
    p = np.arange(pos, pos + m)
    pages = pool[table[b, p // PAGE], :, which]            # [m, hkv, 1152]
    codes = pages[..., :1024].reshape(m, pool.shape[1], 16, 64)[np.arange(m), :, p % PAGE]
    scales = pages[..., 1024:].reshape(m, pool.shape[1], 16, 8)[np.arange(m), :, p % PAGE]
    return decode(codes, scales, g)


def random_tables(rng, need, spare, width=None):
    """(table, pages): scattered pages for sequences of need[b] pages each."""
    pages = sum(need) + spare
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(need), width or max(1, max(need))), -1, np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    return table, pages


class Pages:
    """Page tables, lengths, counts and contents, one operation at a time."""

    def __init__(self, pool, table, S, refs):
        self.pool, self.table, self.S, self.refs, self.error = pool.copy(), table.copy(), S.copy(), refs.copy(), 0

    def _err(self, code):
        self.error = self.error or code

    def _free(self, count):
        ids = np.flatnonzero(self.refs == 0)
        return None if len(ids) < count else list(ids[:count])

    def copy(self, src, dst):
        bad = [not (0 <= s < len(self.refs) and 0 <= d < len(self.refs)) for s, d in zip(src, dst)]
        for i, (s, d) in enumerate(zip(src, dst)):
            if not bad[i]:
                others = [j for j in range(len(dst)) if j != i and 0 <= dst[j] < len(self.refs)
                          and 0 <= src[j] < len(self.refs)]
                if s == d or any(dst[j] == d or src[j] == d for j in others):
                    bad[i] = True
        old = self.pool.copy()
        for i, (s, d) in enumerate(zip(src, dst)):
            if bad[i]:
                self._err(1)
            else:
                self.pool[:, d] = old[:, s]

    def reserve(self, seqs, tokens):
        need = []
        for q, t in zip(seqs, tokens):
            ok = 0 <= q < len(self.S) and 0 <= t <= PAGE * self.table.shape[1] and list(seqs).count(q) == 1
            if ok:
                held = int((self.table[q] >= 0).sum())
                ok = (self.table[q, :held] >= 0).all()
            if not ok:
                self._err(1)
            need.append(max(0, -(-t // PAGE) - held) if ok else 0)
        free = self._free(sum(need))
        if free is None:
            return self._err(4)
        for q, m in zip(seqs, need):
            for _ in range(m):
                page = free.pop(0)
                self.table[q, int((self.table[q] >= 0).sum())] = page
                self.refs[page] = 1

    def fork(self, parents, children):
        ok = []
        for a, c in zip(parents, children):
            good = 0 <= a < len(self.S) and 0 <= c < len(self.S) and list(children).count(c) == 1 \
                and c not in list(parents) and (self.table[c] < 0).all()
            if good:
                L = self.S[a]
                good = 0 <= L <= PAGE * self.table.shape[1]
                if good:
                    mine = self.table[a, :-(-L // PAGE)]
                    good = all(0 <= x < len(self.refs) and self.refs[x] > 0 for x in mine)
            if not good:
                self._err(1)
            ok.append(good)
        free = self._free(sum(1 for a, g in zip(parents, ok) if g and self.S[a] % PAGE))
        if free is None:
            return self._err(4)
        for a, c, good in zip(parents, children, ok):
            if not good:
                continue
            full = self.S[a] // PAGE
            self.table[c, :full] = self.table[a, :full]
            for x in self.table[a, :full]:
                self.refs[x] += 1
            if self.S[a] % PAGE:
                page = free.pop(0)
                self.table[c, full] = page
                self.refs[page] = 1
                self.pool[:, page] = self.pool[:, self.table[a, full]]
            self.S[c] = self.S[a]

    def free(self, seqs):
        for q in seqs:
            if not 0 <= q < len(self.S):
                self._err(1)
                continue
            for x in self.table[q]:
                if x == -1:
                    continue
                if not 0 <= x < len(self.refs) or self.refs[x] <= 0:
                    self._err(1)
                else:
                    self.refs[x] -= 1
            self.table[q] = -1
            self.S[q] = 0

    def compact(self):
        used = np.flatnonzero(self.refs > 0)
        u = len(used)
        movers = [x for x in used if x >= u]
        holes = [x for x in range(u) if self.refs[x] <= 0]
        new = np.full(len(self.refs), -1, np.int32)
        new[used] = used
        for m, h in zip(movers, holes):
            new[m] = h
            self.pool[:, h] = self.pool[:, m]
            self.refs[h], self.refs[m] = self.refs[m], 0
        for at in np.ndindex(*self.table.shape):
            x = self.table[at]
            if x == -1:
                continue
            if not 0 <= x < len(new) or new[x] < 0:
                self._err(1)
            else:
                self.table[at] = new[x]
        return new
