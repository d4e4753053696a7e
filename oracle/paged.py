"""Paged key/value cache and attention over it, in 64 bits and plain loops.

A slow, independent restatement of the definitions in ``include/fa.h`` (fa_cache and the calls on
it), for comparison with the kernels."""
from __future__ import annotations

import numpy as np


class Refused(Exception):
    """A call that the device refuses whole."""


class Pool:
    """Tables, lengths and reference counts of a cache, and the page of every token."""

    def __init__(self, pages, page_size, seqs, seq_pages):
        self.ps, self.width = page_size, seq_pages
        self.table = np.full((seqs, seq_pages), -1, dtype=np.int32)
        self.lens = np.zeros(seqs, dtype=np.int32)
        self.refs = np.zeros(pages, dtype=np.int32)

    def state(self):
        return self.table.copy(), self.lens.copy(), self.refs.copy()

    def _need(self, n):
        return -(-int(n) // self.ps)

    def _free(self, count):
        got = [int(p) for p in np.flatnonzero(self.refs == 0)[:count]]
        if len(got) < count:
            raise Refused("pages")
        return got

    def _slots(self, seqs):
        seqs = [int(s) for s in seqs]
        if any(not 0 <= s < self.lens.size for s in seqs):
            raise Refused("slot")
        return seqs

    def extend(self, seqs, counts):
        seqs = self._slots(seqs)
        if len(set(seqs)) < len(seqs) or any(c < 0 for c in counts):
            raise Refused("list")
        want = [self._need(self.lens[s] + c) for s, c in zip(seqs, counts)]
        if any(w > self.width for w in want):
            raise Refused("length")
        have = [self._need(self.lens[s]) for s in seqs]
        fresh = self._free(sum(want) - sum(have))
        pos = self.lens[seqs].copy()
        for s, a, b, c in zip(seqs, have, want, counts):
            for i in range(a, b):
                self.table[s, i] = fresh.pop(0)
                self.refs[self.table[s, i]] = 1
            self.lens[s] += c
        return pos

    def fork(self, src, dst):
        """Returns the page copies (from, to)."""
        src, dst = self._slots(src), self._slots(dst)
        if len(set(dst)) < len(dst) or set(src) & set(dst) or any(self.lens[d] for d in dst):
            raise Refused("list")
        part = [self.lens[s] % self.ps > 0 for s in src]
        fresh = self._free(sum(part))
        copies = []
        for s, d, p in zip(src, dst, part):
            full = self.lens[s] // self.ps
            self.table[d] = -1
            self.table[d, :full] = self.table[s, :full]
            for q in self.table[s, :full]:
                self.refs[q] += 1
            if p:
                new = fresh.pop(0)
                copies.append((int(self.table[s, full]), new))
                self.table[d, full] = new
                self.refs[new] = 1
            self.lens[d] = self.lens[s]
        return copies

    def free(self, seqs):
        seqs = self._slots(seqs)
        if len(set(seqs)) < len(seqs):
            raise Refused("list")
        for s in seqs:
            for q in self.table[s]:
                if q >= 0:
                    self.refs[q] -= 1
            self.table[s] = -1
            self.lens[s] = 0

    def compact(self):
        live = int((self.refs > 0).sum())
        src = [int(p) for p in np.flatnonzero(self.refs > 0) if p >= live]
        dst = [int(p) for p in np.flatnonzero(self.refs == 0) if p < live]
        for a, b in zip(src, dst):
            self.table[self.table == a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
        return list(zip(src, dst))

    def where(self, slot, j):
        """Page and row of token j."""
        return int(self.table[slot, j // self.ps]), j % self.ps


def copies_refused(pages, src, dst):
    bad = [p for p in list(src) + list(dst) if not 0 <= p < pages]
    return bool(bad) or len(set(dst)) < len(dst) or bool(set(src) & set(dst))


def attend(q, k, v, T, pos0, scale, causal=True, window_left=-1, softcap=0.0):
    """One sequence: q [Hq, T, d] at positions pos0 .. pos0 + T - 1, k and v [Hkv, n, d] dense.
    Returns O, LSE, and per row A = sum p |v| and X = scale * max_j sum |q||k|, in which error
    bounds are stated."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    Hq, _, d = q.shape
    Hkv, n, _ = k.shape
    O, A = np.zeros((Hq, T, d)), np.zeros((Hq, T, d))
    L, X = np.full((Hq, T), -np.inf), np.zeros((Hq, T))
    for h in range(Hq):
        hk = h // (Hq // Hkv)
        for t in range(T):
            i = pos0 + t
            hi = min(n, i + 1) if causal else n
            lo = max(0, i - window_left) if window_left >= 0 else 0
            if hi <= lo:
                continue
            x = scale * (k[hk, lo:hi] @ q[h, t])
            X[h, t] = abs(scale) * (np.abs(k[hk, lo:hi]) @ np.abs(q[h, t])).max()
            if softcap > 0:
                x = softcap * np.tanh(x / softcap)
            m = x.max()
            p = np.exp(x - m)
            z = p.sum()
            L[h, t] = m + np.log(z)
            O[h, t] = p @ v[hk, lo:hi] / z
            A[h, t] = p @ np.abs(v[hk, lo:hi]) / z
    return O, L, A, X
