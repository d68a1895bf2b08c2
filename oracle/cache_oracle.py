"""Plain oracle of the history cache and of the attention that reads it.

TEST INFRASTRUCTURE, like the rest of this package: only the tests import it.

The page bookkeeping is Python integers, one entry after another; the rows are
copied one by one; the attention is fp64 over the rows gathered by position.
"""
from __future__ import annotations

import numpy as np


class CacheModel:
    """The state of a history cache and the rows of one layer's pool.

    A call that the library refuses for an entry leaves that entry undone and
    puts the device bit it sets into `bits` (2: an index or a length that
    cannot be, 4: no room)."""

    def __init__(self, n_pages, page_size, H_kv, d, max_seqs, max_pages):
        self.ps, self.max_pages = page_size, max_pages
        self.table = np.full((max_seqs, max_pages), -1, dtype=np.int32)
        self.lens = np.zeros(max_seqs, dtype=np.int32)
        self.refs = np.zeros(n_pages, dtype=np.int32)
        self.k = np.zeros((n_pages, H_kv, page_size, d), dtype=np.int16)  # bf16 bits
        self.v = np.zeros_like(self.k)
        self.bits = 0

    def pages_of(self, rows):
        return -(-int(rows) // self.ps)

    def _seq(self, s):
        if s >= len(self.lens):
            self.bits |= 2
        return 0 <= s < len(self.lens)

    def fork(self, src, dst):
        pairs = [(s, t) for s, t in zip(src, dst) if s >= 0 and t >= 0]
        targets = [t for _, t in pairs]
        for i, (s, t) in enumerate(pairs):
            if not self._seq(s) or not self._seq(t):
                continue
            if t in targets[:i] or s in targets or self.lens[t] != 0:
                self.bits |= 2
                continue
            n = self.pages_of(self.lens[s])
            self.table[t, :n] = self.table[s, :n]
            self.lens[t] = self.lens[s]
            for p in self.table[s, :n]:
                self.refs[p] += 1

    def free(self, seqs, keep=None):
        seen = set()
        for i, s in enumerate(seqs):
            if s < 0:
                continue
            kept = 0 if keep is None else keep[i]
            if not self._seq(s):
                continue
            if s in seen or kept < 0:
                self.bits |= 2
                seen.add(s)
                continue
            seen.add(s)
            if kept >= self.lens[s]:
                continue
            for slot in range(self.pages_of(kept), self.pages_of(self.lens[s])):
                self.refs[self.table[s, slot]] -= 1
                self.table[s, slot] = -1
            self.lens[s] = kept

    def reserve(self, seqs, counts):
        plan = [[0, 0, -1, -1] for _ in seqs]
        wanted, seen = [], set()  # (entry, slot), in order
        refs0 = self.refs.copy()
        served = []
        for i, (s, c) in enumerate(zip(seqs, counts)):
            if s < 0:
                continue
            if not self._seq(s):
                continue
            if s in seen or c < 0:
                self.bits |= 2
                seen.add(s)
                continue
            seen.add(s)
            n = int(self.lens[s])
            plan[i][0] = n
            if n + c > self.max_pages * self.ps:
                self.bits |= 4
                continue
            if c == 0:
                continue
            slots = list(range(self.pages_of(n), self.pages_of(n + c)))
            cow = -1
            if n % self.ps and refs0[self.table[s, n // self.ps]] > 1:
                cow = int(self.table[s, n // self.ps])
                slots.insert(0, n // self.ps)
            served.append((i, s, c, cow))
            wanted += [(i, s, slot) for slot in slots]
        free = np.nonzero(refs0 == 0)[0]
        if len(wanted) > len(free):
            self.bits |= 4
            return plan
        for (i, s, slot), p in zip(wanted, free):
            self.table[s, slot] = p
            self.refs[p] = 1
        for i, s, c, cow in served:
            plan[i][1] = c
            if cow >= 0:
                self.refs[cow] -= 1
                plan[i][2] = cow
                plan[i][3] = int(self.table[s, plan[i][0] // self.ps])
            self.lens[s] += c
        return plan

    def write(self, seqs, plan, k_new, v_new):
        """k_new, v_new: bf16 bits [n, H_kv, L, d]."""
        for i, s in enumerate(seqs):
            if s < 0:
                continue
            first, count, old, new = plan[i]
            for pages, rows in ((self.k, k_new), (self.v, v_new)):
                if old >= 0:
                    for at in range(first % self.ps):
                        pages[new, :, at] = pages[old, :, at]
                for j in range(count):
                    pos = first + j
                    pages[self.table[s, pos // self.ps], :, pos % self.ps] = rows[i, :, j]

    def compact(self):
        """Renumbers the pages and moves their rows; the list of (from, to)."""
        live = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        M = len(live)
        holes = [p for p in range(M) if self.refs[p] == 0]
        moves = list(zip([p for p in live if p >= M], holes))
        for a, b in moves:
            self.table[self.table == a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.k[b], self.v[b] = self.k[a], self.v[a]
        return moves

    def check(self):
        """The counts are what the table says, and entries past a sequence's end are empty."""
        want = np.zeros_like(self.refs)
        for s, n in enumerate(self.lens):
            used = self.pages_of(n)
            for p in self.table[s, :used]:
                want[p] += 1
            assert np.all(self.table[s, used:] == -1)
        assert np.array_equal(want, self.refs)


def gather_rows(pages, entries, lo, hi, page_size):
    """Rows at positions [lo, hi) of a sequence with page numbers `entries`: [H_kv, hi - lo, d]."""
    at = np.arange(lo, hi)
    return np.moveaxis(pages[np.asarray(entries)[at // page_size], :, at % page_size], 0, 1)


def prefix_attention(q, k, v, table, lens, seqs, prefix_seq, prefix_len, scale, page_size):
    """(O, lse, spread) of svg_prefix_attention in fp64; spread = sum_j w_j |v_j|, what a
    relative error of every weight can move O by. q [B, H, Lq, d]; k, v pools (values).
    Entries with a negative sequence get NaN."""
    B, H, Lq, d = q.shape
    G = H // k.shape[1]
    o, spread = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse = np.full(q.shape[:3], np.nan)
    for b, s in enumerate(seqs):
        if s < 0:
            continue
        kk = [gather_rows(x, table[prefix_seq], 0, prefix_len, page_size) for x in (k, v)]
        own = [gather_rows(x, table[s], prefix_len, max(prefix_len, lens[s]), page_size)
               for x in (k, v)]
        ks, vs = (np.concatenate(x, axis=1) for x in zip(kk, own))
        for h in range(H):
            if ks.shape[1] == 0:
                o[b, h], spread[b, h], lse[b, h] = 0.0, 0.0, -np.inf
                continue
            x = scale * (q[b, h] @ ks[h // G].T)
            m = x.max(axis=1, keepdims=True)
            w = np.exp(x - m)
            t = w.sum(axis=1, keepdims=True)
            o[b, h] = w @ vs[h // G] / t
            spread[b, h] = w @ np.abs(vs[h // G]) / t
            lse[b, h] = (m + np.log(t))[:, 0]
    return o, lse, spread
