"""fp64 CPU oracle of the attention window's operators: rotary positions, the
paged 8-bit cache as a model of plain Python lists, and the attention over it.

TEST INFRASTRUCTURE ONLY: imported by the tests, never by the product
library.  It shares no code with the HIP path.  What it computes is stated in
include/tm_attention.h.
"""
from __future__ import annotations

import numpy as np

PAGE, BLOCK = 64, 16
E_MIN, E_MAX = -110, 119
NONFINITE, NO_PAGES, FULL, BAD_ENTRY = 1, 2, 4, 8


def rotate(x, positions, freq, scale=1.0, interleaved=False, inverse=False):
    """x [B][T][H][d], positions [B][T] -> rotated, fp64 (angles in extended
    precision)."""
    x = np.asarray(x, np.float64)
    n = len(freq)
    angle = np.asarray(positions, np.longdouble)[..., None] * np.asarray(freq, np.longdouble)
    cos, sin = (np.asarray(f(angle), np.float64)[:, :, None] for f in (np.cos, np.sin))
    if inverse:
        sin = -sin
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    ya, yb = scale * (a * cos - b * sin), scale * (a * sin + b * cos)
    y = x.copy()
    if interleaved:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = ya, yb
    else:
        y[..., :n], y[..., n:2 * n] = ya, yb
    return y


def exponent(amax):
    """The least e in [E_MIN, E_MAX] with amax <= 448 2^e."""
    e = E_MIN
    while e < E_MAX and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def round_e4m3(x):
    """fp64 -> the nearest e4m3 value (ties to even, 448 the largest)."""
    x = np.clip(np.asarray(x, np.float64), -448.0, 448.0)
    _, e = np.frexp(x)                                   # |x| in [2^(e-1), 2^e): steps of 2^(e-4), 2^-9 at least
    step = 2.0 ** np.maximum(e - 4, -9)
    return np.round(x / step) * step


class Cache:
    """The cache's rules, one token at a time.  A page: codes (as values)
    and exponents of keys and values."""

    def __init__(self, kv_heads, head_dim, n_pages, n_seqs, seq_pages):
        self.H, self.d, self.seq_pages = kv_heads, head_dim, seq_pages
        self.codes = np.zeros((n_pages, 2, kv_heads, PAGE, head_dim))
        self.exps = np.zeros((n_pages, 2, kv_heads, PAGE // BLOCK), np.int64)
        self.refs = [0] * n_pages
        self.pages = [[] for _ in range(n_seqs)]         # each sequence's pages
        self.lengths = [0] * n_seqs
        self.flags = 0

    def used(self):
        return sum(r > 0 for r in self.refs)

    def append(self, seqs, counts, k, v):
        """k, v [B][T][H][d] (fp32 or bf16 values)."""
        free = [p for p, r in enumerate(self.refs) if r == 0]
        before, asked, seen, todo = list(self.refs), 0, set(), []
        for b, s in enumerate(seqs):
            if not 0 <= s < len(self.lengths) or s in seen:
                self.flags |= BAD_ENTRY
                continue
            seen.add(s)
            n, old = min(max(counts[b], 0), k.shape[1]), self.lengths[s]
            if old + n > self.seq_pages * PAGE:
                self.flags |= FULL
                continue
            if n == 0:
                continue
            shared = old % PAGE > 0 and before[self.pages[s][-1]] > 1
            need = -(-(old + n) // PAGE) - -(-old // PAGE) + shared
            first, asked = asked, asked + need
            if need and asked > len(free):
                self.flags |= NO_PAGES
                continue
            todo.append((b, s, n, shared, free[first:asked]))
        for b, s, n, shared, new in todo:
            for p in new:
                self.refs[p] = 1
            if shared:
                src, dst = self.pages[s][-1], new[0]
                self.codes[dst], self.exps[dst] = self.codes[src], self.exps[src]
                self.refs[src] -= 1
                self.pages[s][-1] = dst
                new = new[1:]
            self.pages[s] = self.pages[s] + new
            for w, x in enumerate((k, v)):
                self._write(s, w, self.lengths[s], np.asarray(x[b, :n], np.float64))
            self.lengths[s] += n

    def _write(self, s, w, at, x):
        good = np.isfinite(x)
        if not good.all():
            self.flags |= NONFINITE
        x = np.where(good, x, 0.0)
        t = 0
        while t < len(x):
            p, o = self.pages[s][(at + t) // PAGE], (at + t) % PAGE
            n = min(BLOCK - o % BLOCK, len(x) - t)
            for h in range(self.H):
                new = x[t:t + n, h]
                e = exponent(np.abs(new).max())
                if o % BLOCK:
                    had = int(self.exps[p, w, h, o // BLOCK])
                    e = max(e, had)
                    lo = o // BLOCK * BLOCK
                    self.codes[p, w, h, lo:o] = round_e4m3(self.codes[p, w, h, lo:o] * 2.0 ** (had - e))
                self.exps[p, w, h, o // BLOCK] = e
                self.codes[p, w, h, o:o + n] = round_e4m3(new * 2.0 ** -e)
            t += n

    def fork(self, src, dst):
        lengths = list(self.lengths)
        for i, (s, d) in enumerate(zip(src, dst)):
            n = len(lengths)
            if not (0 <= s < n and 0 <= d < n) or d in dst[:i] or s in dst or lengths[d] != 0:
                self.flags |= BAD_ENTRY
                continue
            self.pages[d] = list(self.pages[s])
            self.lengths[d] = lengths[s]
            for p in self.pages[d]:
                self.refs[p] += 1

    def free(self, seqs, keep=None):
        for i, s in enumerate(seqs):
            if not 0 <= s < len(self.lengths) or s in seqs[:i]:
                self.flags |= BAD_ENTRY
                continue
            n = 0 if keep is None else min(max(keep[i], 0), self.lengths[s])
            left = -(-n // PAGE)
            for p in self.pages[s][left:]:
                self.refs[p] -= 1
            self.pages[s] = self.pages[s][:left]
            self.lengths[s] = n

    def compact(self):
        n = self.used()
        src = [p for p, r in enumerate(self.refs) if r > 0 and p >= n]
        dst = [p for p, r in enumerate(self.refs) if r == 0 and p < n]
        to = dict(zip(src, dst))
        for a, b in to.items():
            self.codes[b], self.exps[b], self.refs[b], self.refs[a] = self.codes[a], self.exps[a], self.refs[a], 0
        self.pages = [[to.get(p, p) for p in ps] for ps in self.pages]

    def held(self, s):
        """(k, v) [tokens][H][d]: the values a sequence's tokens are held as."""
        n = self.lengths[s]
        out = []
        for w in range(2):
            x = np.zeros((n, self.H, self.d))
            for t in range(n):
                p, o = self.pages[s][t // PAGE], t % PAGE
                x[t] = self.codes[p, w, :, o] * 2.0 ** self.exps[p, w, :, o // BLOCK][:, None]
            out.append(x)
        return out

    def attend(self, s, q, scale, window=0, sink=0):
        return attend(*self.held(s), q, scale, window, sink)


def visible(length, count, window=0, sink=0):
    """[count][length]: which tokens the last `count` of a sequence see."""
    pos = length - count + np.arange(count)[:, None]
    j = np.arange(length)[None]
    see = j <= pos
    if window:
        see &= (j > pos - window) | (j < sink)
    return see


def attend(k, v, q, scale, window=0, sink=0):
    """k, v [L][H][d], q [count][heads][d] (fp64) -> (out [count][heads][d],
    spread: the weighted mean of |v|, score error: scale times the largest
    sum |q||k| that a row sees), the last two for error bounds."""
    L, H, d = k.shape
    n, heads, _ = q.shape
    see = visible(L, n, window, sink)
    out, spread, size = np.zeros((n, heads, d)), np.zeros((n, heads, d)), np.zeros((n, heads, 1))
    for g in range(heads):
        h = g // (heads // H)
        s = scale * (q[:, g] @ k[:, h].T)
        size[:, g, 0] = np.where(see, abs(scale) * (np.abs(q[:, g]) @ np.abs(k[:, h]).T), 0).max(axis=1, initial=0)
        s = np.where(see, s, -np.inf)
        top = s.max(axis=1, initial=-np.inf, keepdims=True)
        p = np.exp(s - np.where(np.isfinite(top), top, 0))
        total = p.sum(axis=1, keepdims=True)
        p /= np.where(total > 0, total, 1)
        out[:, g], spread[:, g] = p @ v[:, h], p @ np.abs(v[:, h])
    return out, spread, size
