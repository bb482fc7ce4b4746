"""References of the 4-bit cache, its pages and the rotation, in float64 and
plain Python (no product code): what include/hga.h says, done one thing at a
time."""
import math

import numpy as np

MAG = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
SCALES = np.array([(m * 2.0 ** -17) if e == 0 else (1 + m / 8) * 2.0 ** (e - 15)
                   for e in range(29) for m in range(8)][:227])


def stored(x):
    """Values that the cache keeps of x [..., d] (d a multiple of 16), float64."""
    f = np.asarray(x, dtype=np.float64)
    f = np.where(np.isnan(f), 0.0, f)
    f = np.clip(f, -61440.0, 61440.0).reshape(f.shape[:-1] + (-1, 16))
    top = np.abs(f).max(-1)
    b = np.searchsorted(6 * SCALES, top)              # first scale that is large enough
    s = SCALES[b][..., None]
    r = np.abs(f) / np.where(s > 0, s, 1.0)
    hi = np.minimum(np.searchsorted(MAG, r), 7)
    lo = np.maximum(hi - 1, 0)
    up, down = MAG[hi] - r, r - MAG[lo]
    idx = np.where(up < down, hi, np.where(up > down, lo, np.where(hi % 2 == 0, hi, lo)))
    return (MAG[idx] * np.sign(f) * s).reshape(np.shape(x))


def attention(q, k, v, allowed):
    """q [r][d], k, v [t][d], allowed [r][t] bool: output, lse, the weighted
    |v|, the largest sum |q k| / sqrt(d) of each row and the unweighted |v|
    relative to the weights' sum; empty rows 0 and -inf."""
    d = q.shape[-1]
    s = q @ k.T / math.sqrt(d)
    s = np.where(allowed, s, -np.inf)
    m = s.max(-1, keepdims=True, initial=-np.inf)
    m = np.where(np.isneginf(m), 0.0, m)
    e = np.exp(s - m)
    l = e.sum(-1, keepdims=True)
    p = e / np.where(l > 0, l, 1.0)
    v = np.where(allowed.any(0)[:, None], v, 0.0)
    with np.errstate(divide="ignore"):
        lse = np.log(l[:, 0]) + m[:, 0]
    mag = np.where(allowed, np.abs(q) @ np.abs(k).T, 0.0).max(-1, initial=0.0) / math.sqrt(d)
    return p @ v, lse, p @ np.abs(v), mag, allowed / np.maximum(l, 1.0) @ np.abs(v)


def tolerance(dtype, o, mag_v, mag_s, all_v, tc=False):
    """Bounds of |kernel - reference| for o and lse, from the arithmetic.

    Score: products of exact fp16 values (fp32 q: two fp16 parts, 22 bits)
    summed in fp32, at most 16 accumulations and as many roundings inside a
    product step, each 2^-23 of the sum of magnitudes: es = 40 * 2^-23 * mag_s.
    The exponent's argument s * scale - max is rounded once more (2^-23 of
    |s| <= mag_s, in both) and 2^x is good to 2^-22.  A weight is off by that in
    its numerator and in the sum, so 2 (es + 2^-21); P is rounded to fp16 (2^-11; fp32: two
    parts, 2^-21), sums of P V add 2^-20.  The output is rounded once.
    P is 2^11 e, e relative to a maximum at most the largest score.  What is
    below fp16's smallest normal value is held to a multiple of 2^-24, so every
    weight may be off by 2^-25 too: 2^-36 all_v.
    tc, the kernel for many query rows: P is 2^7 e, so 2^-32 all_v; 6 of 16
    exponentials are a polynomial good to 7.8e-5, in numerator and sum."""
    out = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}[dtype]
    p = {"bf16": 2.0 ** -11, "fp32": 2.0 ** -21}[dtype]
    es = 42 * 2.0 ** -23 * mag_s
    poly, small = (7.8e-5, 2.0 ** -32) if tc else (0.0, 2.0 ** -36)
    rel = 2 * (es + 2.0 ** -21 + poly) + p + 2.0 ** -20
    to = (rel[..., None] * mag_v + small * all_v) * (1 + out) + out * np.abs(o) + 1e-30
    return to, 2 * es + poly + 2.0 ** -20 + 2.0 ** -22 * 40


def rotate(x, pos, freq, axis, adjacent, sign=1):
    """x [n][heads][d] float64, pos [axes][n]."""
    half = len(freq)
    ang = sign * pos[axis].T.astype(np.float64) * freq          # [n][half]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    y = x.copy()
    a = slice(0, 2 * half, 2) if adjacent else slice(0, half)
    b = slice(1, 2 * half, 2) if adjacent else slice(half, 2 * half)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


class Pool:
    """Bookkeeping of a page pool, one entry after another.  bad counts what
    was refused."""

    def __init__(self, n_planes, n_pages, page_bytes, page_tokens, n_rows, row_pages, rng):
        self.data = rng.integers(0, 256, (n_planes, n_pages, page_bytes), dtype=np.uint8)
        self.table = np.full((n_rows, row_pages), -1, np.int32)
        self.len = np.zeros(n_rows, np.int32)
        self.ref = np.zeros(n_pages, np.int32)
        self.pt, self.bad = page_tokens, 0

    def _free(self):
        return [i for i in range(len(self.ref)) if self.ref[i] == 0]

    def _grant(self, wants):
        """wants: (entry, pages) in order -> pages of each entry, None where they ran out."""
        free, out, used = self._free(), {}, 0
        for i, n in wants:
            used += n
            if n and used > len(free):
                out[i] = None
            else:
                out[i] = free[used - n:used]
        return out

    def reserve(self, rows, new_len):
        seen, wants = set(), []
        for i, (r, n) in enumerate(zip(rows, new_len)):
            if r < 0:
                continue
            first = r not in seen
            seen.add(r)
            if not (r < len(self.len) and first and n >= self.len[r]
                    and n <= self.table.shape[1] * self.pt):
                self.bad += 1
                continue
            wants.append((i, -(-int(n) // self.pt) - -(-int(self.len[r]) // self.pt)))
        for i, pages in self._grant(wants).items():
            if pages is None:
                self.bad += 1
                continue
            r = rows[i]
            at = -(-int(self.len[r]) // self.pt)
            self.table[r, at:at + len(pages)] = pages
            self.ref[pages] = 1
            self.len[r] = new_len[i]

    def fork(self, parents, children):
        kids = {c for c in children if 0 <= c < len(self.len)}
        seen, wants = set(), []
        for i, (p, c) in enumerate(zip(parents, children)):
            if c < 0:
                continue
            first = c not in seen
            seen.add(c)
            if not (c < len(self.len) and 0 <= p < len(self.len) and first and p not in kids
                    and self.len[c] == 0):
                self.bad += 1
                continue
            wants.append((i, int(self.len[p] % self.pt > 0)))
        for i, pages in self._grant(wants).items():
            if pages is None:
                self.bad += 1
                continue
            p, c = parents[i], children[i]
            full = self.len[p] // self.pt
            self.table[c, :full] = self.table[p, :full]
            for pg in self.table[p, :full]:
                self.ref[pg] += 1
            if pages:
                self.table[c, full] = pages[0]
                self.ref[pages[0]] = 1
                self.data[:, pages[0]] = self.data[:, self.table[p, full]]
            self.len[c] = self.len[p]

    def free(self, rows):
        for r in rows:
            if r < 0:
                continue
            if r >= len(self.len):
                self.bad += 1
                continue
            for pg in self.table[r]:
                if pg >= 0:
                    self.ref[pg] -= 1
            self.table[r] = -1
            self.len[r] = 0

    def compact(self):
        used = int((self.ref > 0).sum())
        src = [i for i in range(used, len(self.ref)) if self.ref[i] > 0]
        dst = [i for i in range(used) if self.ref[i] == 0]
        for s, d in zip(src, dst):
            self.data[:, d] = self.data[:, s]
            self.table[self.table == s] = d
            self.ref[d], self.ref[s] = self.ref[s], 0

    def copy(self, src, dst):
        sources = {s for s, d in zip(src, dst) if d >= 0}
        seen = set()
        old = self.data.copy()
        for s, d in zip(src, dst):
            if s < 0 and d < 0:
                continue
            n = len(self.ref)
            first = d not in seen
            seen.add(d)
            if not (0 <= s < n and 0 <= d < n and first and d not in sources):
                self.bad += 1
                continue
            self.data[:, d] = old[:, s]
