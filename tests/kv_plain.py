"""A plain paged e4m3 key/value cache in NumPy: fp64 arithmetic, one token, page and sequence at a time.

Written from the definitions alone: e4m3 from its bit fields, rounding by search in the table of values, block scales
from logarithms corrected by comparison, attention as the sum over visible positions.
"""
import math

import numpy as np


def e4m3_table():
    out = np.empty(256)
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        v = math.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[b] = -v if s else v
    return out


TABLE = e4m3_table()
POS = TABLE[:127]                      # 0 .. 448 ascending


def encode(x):
    """Nearest code (ties to the even one), saturated to +-448; NaN stays NaN."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0, x)), 448.0)
    hi = np.clip(np.searchsorted(POS, a), 1, 126)
    lo = hi - 1
    d_lo, d_hi = a - POS[lo], POS[hi] - a
    c = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi)
    c = c | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), (c & 128) | 127, c).astype(np.uint8)


def block_scale(a):
    if a == 0:
        return 2.0 ** -120
    e = math.ceil(math.log2(a / 448.0))
    while a > 448.0 * 2.0 ** e:
        e += 1
    while a <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    return 2.0 ** max(e, -120)


class PlainCache:
    def __init__(self, n_layers, hq, hkv, dim, page, n_pages, max_seqs, max_pages, rng=None):
        """rng: fill the pool with random bytes (NaN codes among them) and NaN scales: what nothing may read."""
        self.hq, self.hkv, self.dim, self.page, self.n_pages = hq, hkv, dim, page, n_pages
        shape = (n_layers, n_pages, hkv, page, dim)
        self.k = np.zeros(shape, np.uint8) if rng is None else rng.integers(0, 256, shape).astype(np.uint8)
        self.v = self.k[..., ::-1].copy()
        self.ks = np.full(shape[:3], 0.0 if rng is None else math.nan)
        self.vs = self.ks.copy()
        self.table = np.full((max_seqs, max_pages), -1, np.int32)
        self.length = np.zeros(max_seqs, np.int32)
        self.ref = np.zeros(n_pages, np.int32)
        self.oom = False

    def pages(self, length):
        return -(-int(length) // self.page)

    def take(self, n):
        got = np.flatnonzero(self.ref == 0)[:n]
        if len(got) < n:
            return None
        self.ref[got] = 1
        return got

    def reserve(self, seqs, new):
        short = False
        for s, n in zip(seqs, new):
            have, want = self.pages(self.length[s]), self.pages(self.length[s] + n)
            if self.length[s] + n > self.table.shape[1] * self.page:
                self.oom = True
                continue
            if want > have:
                got = None if short else self.take(want - have)
                if got is None:
                    self.oom = short = True
                    continue
                self.table[s, have:want] = got
            self.length[s] += n

    def append(self, layer, seqs, new, k_new, v_new):
        for codes, scales, x in ((self.k, self.ks, k_new), (self.v, self.vs, v_new)):
            x = np.asarray(x, np.float64)
            row = 0
            for s, n in zip(seqs, new):
                total = int(self.length[s])
                at = total - n
                while at < total:
                    c = at // self.page
                    end, old, page = min(total, (c + 1) * self.page), at - c * self.page, self.table[s, c]
                    for h in range(self.hkv):
                        blk = x[row:row + end - at, h]
                        fin = np.abs(blk[np.isfinite(blk)])
                        sc = block_scale(fin.max() if fin.size else 0.0)
                        if old:
                            was = scales[layer, page, h]
                            sc = max(sc, was)
                            if sc > was:
                                codes[layer, page, h, :old] = encode(TABLE[codes[layer, page, h, :old]] * (was / sc))
                        scales[layer, page, h] = sc
                        codes[layer, page, h, old:old + end - at] = encode(blk / sc)
                    row += end - at
                    at = end

    def release(self, s):
        for c in range(self.pages(self.length[s])):
            if self.table[s, c] >= 0:
                self.ref[self.table[s, c]] -= 1
        self.table[s] = -1
        self.length[s] = 0

    free = release

    def copy(self, a, b):
        for x in (self.k, self.v, self.ks, self.vs):
            x[:, b] = x[:, a]

    def fork(self, src, dst):
        for d in dst:
            self.release(d)
        for s, d in zip(src, dst):
            n = int(self.length[s])
            if n % self.page:
                got = self.take(1)
                if got is None:
                    self.oom = True
                    continue
                self.copy(self.table[s, n // self.page], got[0])
                self.table[d, n // self.page] = got[0]
            full = n // self.page
            self.table[d, :full] = self.table[s, :full]
            for p in self.table[s, :full]:
                if p >= 0:
                    self.ref[p] += 1
            self.length[d] = n

    def trim(self, s, window, sinks):
        for c in range(self.pages(self.length[s])):
            if c * self.page >= sinks and (c + 1) * self.page - 1 <= self.length[s] - window and self.table[s, c] >= 0:
                self.ref[self.table[s, c]] -= 1
                self.table[s, c] = -1

    def compact(self):
        m = int((self.ref > 0).sum())
        for a, b in zip([p for p in range(m, self.n_pages) if self.ref[p] > 0],
                        [p for p in range(m) if self.ref[p] == 0]):
            self.copy(a, b)
            self.ref[b], self.ref[a] = self.ref[a], 0
            self.table[self.table == a] = b
        return m

    def attend(self, layer, seqs, new, q, scale, window=0, sinks=0):
        """(out, lse) in fp64."""
        q = np.asarray(q, np.float64)
        out, lse = np.zeros(q.shape), np.full(q.shape[:2], -math.inf)
        group, row = self.hq // self.hkv, 0
        for s, n in zip(seqs, new):
            total = int(self.length[s])
            j = np.arange(total)
            page = self.table[s, j // self.page]
            j, page = j[page >= 0], page[page >= 0]
            for t in range(n):
                pos = total - n + t
                see = j <= pos
                if window > 0:
                    see &= (pos - j < window) | (j < sinks)
                jj, pp = j[see], page[see]
                if jj.size:
                    for h in range(self.hkv):
                        k = TABLE[self.k[layer, pp, h, jj % self.page]] * self.ks[layer, pp, h][:, None]
                        v = TABLE[self.v[layer, pp, h, jj % self.page]] * self.vs[layer, pp, h][:, None]
                        x = q[row, h * group:(h + 1) * group] @ k.T * scale
                        top = x.max(-1, keepdims=True)
                        p = np.exp(x - top)
                        z = p.sum(-1, keepdims=True)
                        out[row, h * group:(h + 1) * group] = (p / z) @ v
                        lse[row, h * group:(h + 1) * group] = (top + np.log(z))[:, 0]
                row += 1
        return out, lse
