"""Plain float64 statement of the paged cache and of the tree decodes over it.

TEST INFRASTRUCTURE ONLY, like fib_oracle.py: it shares no code with the CUDA path.  The cache's
calls are written one sequence after the other, in the order that include/fib_attn.h states; the
decodes build each node's keys one by one from its line of ancestors.
"""
from __future__ import annotations

import math

import numpy as np


def turn(x: np.ndarray, pos, rope_base: float = 10000.0) -> np.ndarray:
    """RoPE (rotate-half pairs (m, m + D/2)) of x [..., D] at positions `pos`, broadcast over x[..., 0]."""
    h = x.shape[-1] // 2
    a = np.asarray(pos, np.float64)[..., None] * rope_base ** (-np.arange(h) / h)
    c, s = np.cos(a), np.sin(a)
    return np.concatenate([x[..., :h] * c - x[..., h:] * s, x[..., :h] * s + x[..., h:] * c], axis=-1)


class PagedCache:
    """Tables, counts and rows of a cache; k and v [layers, pages, heads, P, D], float64."""

    def __init__(self, k, v, table, lens, refs):
        self.k, self.v = k, v
        self.P = k.shape[3]
        self.table, self.lens, self.refs = [list(r) for r in table], list(lens), list(refs)

    def pages(self, n: int) -> int:
        return -(-n // self.P)

    def commit(self, k_new, v_new, n_new, path=None, rnd=lambda x: x) -> bool:
        """Rows of accepted nodes; False (and nothing done) where the pages do not suffice."""
        P, holders = self.P, {}
        for b, n in enumerate(n_new):
            if n and self.lens[b] % P:
                holders.setdefault(self.table[b][self.lens[b] // P], []).append(b)
        copies = []
        for page, seqs in holders.items():
            if self.refs[page] > 1:
                keeper = max(seqs, key=lambda b: (self.lens[b], b)) if len(seqs) == self.refs[page] else None
                copies += [b for b in seqs if b != keeper]
        fresh = [self.pages(self.lens[b] + n) - self.pages(self.lens[b]) if n else 0 for b, n in enumerate(n_new)]
        free = [p for p, c in enumerate(self.refs) if c == 0]
        if len(copies) + sum(fresh) > len(free):
            return False
        before = self.k.copy(), self.v.copy()
        for b, n in enumerate(n_new):
            j, rows = divmod(self.lens[b], P)
            if b in copies:
                old, new = self.table[b][j], free.pop(0)
                self.k[:, new, :, :rows], self.v[:, new, :, :rows] = before[0][:, old, :, :rows], before[1][:, old, :, :rows]
                self.refs[old] -= 1
                self.refs[new] = 1
                self.table[b][j] = new
            first = self.pages(self.lens[b])
            for i in range(fresh[b]):
                self.table[b][first + i] = free.pop(0)
                self.refs[self.table[b][first + i]] = 1
            for i in range(n):
                p = self.lens[b] + i
                node = i if path is None else path[b][i]
                at = self.table[b][p // P]
                self.k[:, at, :, p % P] = rnd(turn(k_new[:, b, :, node], p))
                self.v[:, at, :, p % P] = v_new[:, b, :, node]
            self.lens[b] += n
        return True

    def fork(self, src):
        old_t, old_l = [list(r) for r in self.table], list(self.lens)
        for b, s in enumerate(src):
            if s == b:
                continue
            held = self.pages(old_l[b])
            for j in range(held):
                self.refs[old_t[b][j]] -= 1
                self.table[b][j] = -1
            self.lens[b] = old_l[s] if s >= 0 else 0
            for j in range(self.pages(self.lens[b])):
                self.table[b][j] = old_t[s][j]
                self.refs[old_t[s][j]] += 1

    def compact(self):
        n = sum(c > 0 for c in self.refs)
        holes = [p for p in range(n) if self.refs[p] == 0]
        remap = [p if c > 0 else -1 for p, c in enumerate(self.refs)]
        for p in range(n, len(self.refs)):
            if self.refs[p] > 0:
                to = holes.pop(0)
                self.k[:, to], self.v[:, to] = self.k[:, p], self.v[:, p]
                self.refs[to], self.refs[p], remap[p] = self.refs[p], 0, to
        for b, row in enumerate(self.table):
            for j in range(self.pages(self.lens[b])):
                row[j] = remap[row[j]]
        return remap, n

    def rows(self, layer: int, b: int):
        """K and V of sequence b as [len, heads, D]."""
        p = np.arange(self.lens[b])
        page = np.asarray(self.table[b])[p // self.P].astype(int)
        return self.k[layer, page, :, p % self.P], self.v[layer, page, :, p % self.P]


def tree_attend(cache: PagedCache, layer: int, q, k_new, v_new, parent, n_nodes, keys=None):
    """(o, lse) of every live node; q [B, Hq, T, D], k_new, v_new [B, H, T, D] raw.  keys: [(lo, w)] of
    the layer's window and rungs, or None: every key (dense).  Rows of padding stay NaN."""
    B, Hq, T, D = q.shape
    G = Hq // k_new.shape[1]
    o, lse = np.full(q.shape, np.nan), np.full(q.shape[:3], np.nan)
    for b in range(B):
        K, V = cache.rows(layer, b)
        n = cache.lens[b]
        for s in range(n_nodes[b]):
            line = [s]  # the node and its ancestors, nearest first
            while parent[b][line[-1]] >= 0:
                line.append(parent[b][line[-1]])
            pos = n + len(line) - 1
            kl = np.stack([turn(k_new[b, :, u], pos - i) for i, u in enumerate(line)])  # [line, H, D]
            ks = np.concatenate([kl, K[::-1]])  # by distance
            vs = np.concatenate([v_new[b][:, line].transpose(1, 0, 2), V[::-1]])
            if keys is not None:
                live = [(lo, w) for lo, w in keys if lo + (w > 0) <= pos]
                ks = np.stack([(1 - w) * ks[lo] + w * ks[lo + 1] if w > 0 else ks[lo] for lo, w in live])
                vs = np.stack([(1 - w) * vs[lo] + w * vs[lo + 1] if w > 0 else vs[lo] for lo, w in live])
            for h in range(Hq):
                sc = ks[:, h // G] @ turn(q[b, h, s], pos) / math.sqrt(D)
                m = sc.max()
                p = np.exp(sc - m)
                lse[b, h, s] = m + math.log(p.sum())
                o[b, h, s] = p @ vs[:, h // G] / p.sum()
    return o, lse
