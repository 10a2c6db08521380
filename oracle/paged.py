"""Paged 8-bit key/value cache in plain NumPy: e4m3, appending with rotation, attention.

Written from the definitions alone, one sequence, page, head and token at a time. The attention is in
float64. The append rounds each product and sum of the rotation to float32, as its definition says, so
that codes and scales can be compared bit for bit; ``dtype=numpy.float64`` gives the unrounded rotation.
"""

import math

import numpy as np


def _values():
    v = np.zeros(256)
    for x in range(256):
        e, f = (x >> 3) & 15, x & 7
        a = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v[x] = (math.nan if (x & 127) == 127 else a) * (-1 if x & 128 else 1)
    return v


E4M3 = _values()           # value of each code
_POSITIVE = E4M3[:127]     # ascending: 0 .. 448


def encode(x):
    """e4m3 codes of an array: nearest, halves to the even code, above 448 to 448, NaN to NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    up = np.searchsorted(_POSITIVE, a, side="left").clip(1, 126)
    lo, hi = _POSITIVE[up - 1], _POSITIVE[up]
    mid = (lo + hi) / 2
    code = np.where(a < mid, up - 1, np.where(a > mid, up, np.where(up % 2 == 0, up, up - 1)))
    code = np.where(a >= 448, 126, code)
    code = np.where(np.isnan(x), 127, code)
    return (code | (np.signbit(x).astype(np.int64) << 7)).astype(np.uint8)


def scale_of(amax):
    """Smallest power of two s >= 2^-126 with amax / s <= 448; 1 for 0."""
    if amax == 0:
        return 1.0
    m, e = math.frexp(float(amax))
    return 2.0 ** max(e - (9 if m <= 0.875 else 8), -126)


def rotate(x, cos, sin, interleaved, dtype=np.float32):
    """x [..., d] with the angles of its position; cos, sin [rot / 2]."""
    y = np.array(x, dtype=dtype)
    h = len(cos)
    c, s = np.asarray(cos, dtype=dtype), np.asarray(sin, dtype=dtype)
    ia = np.arange(h) * 2 if interleaved else np.arange(h)
    ib = ia + 1 if interleaved else ia + h
    a, b = y[..., ia].copy(), y[..., ib].copy()
    with np.errstate(invalid="ignore", over="ignore"):
        y[..., ia] = a * c - b * s
        y[..., ib] = b * c + a * s
    return y


class Cache:
    """A pool with the operators on it; pages are uint8 codes [P, H, page, d]."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        self.codes = {"k": np.array(k_codes, dtype=np.uint8), "v": np.array(v_codes, dtype=np.uint8)}
        self.scales = {"k": np.array(k_scales, dtype=np.float64), "v": np.array(v_scales, dtype=np.float64)}
        self.page = self.codes["k"].shape[2]

    def _write(self, name, x, old, length, pages):
        """x [n, H, d]: the tokens at positions [old, length) of a sequence with these pages."""
        page = self.page
        for idx in range(old // page, -(-length // page)):
            lo, hi = max(old, idx * page), min(length, (idx + 1) * page)
            p = pages[idx]
            for h in range(x.shape[1]):
                new = np.asarray(x[lo - old:hi - old, h], dtype=np.float64)
                fine = np.abs(new[np.isfinite(new)])
                s = scale_of(fine.max() if fine.size else 0.0)
                held = lo - idx * page
                if held:
                    was = self.scales[name][p, h]
                    s = max(s, was)
                    if s > was:
                        block = self.codes[name][p, h, :held]
                        self.codes[name][p, h, :held] = encode(E4M3[block] * (was / s))
                self.scales[name][p, h] = s
                self.codes[name][p, h, held:held + hi - lo] = encode(new / s)

    def append(self, table, lens, cu, k, v, cos=None, sin=None, interleaved=False, dtype=np.float32):
        """k, v [T, H, d]; the rows of sequence b are cu[b] .. cu[b + 1]."""
        for b, length in enumerate(lens):
            n = cu[b + 1] - cu[b]
            skip = max(n - length, 0)
            rows = range(cu[b] + skip, cu[b + 1])
            if not len(rows):
                continue
            old = length - len(rows)
            kk = np.stack([k[r] if cos is None else rotate(k[r], cos[old + i], sin[old + i], interleaved, dtype)
                           for i, r in enumerate(rows)])
            self._write("k", kk, old, length, table[b])
            self._write("v", np.stack([v[r] for r in rows]), old, length, table[b])

    def read(self, name, pages, length):
        """The first `length` cached values of a sequence, [H, length, d]."""
        ids = list(pages[:-(-length // self.page)])
        x = E4M3[self.codes[name][ids]] * self.scales[name][ids][..., None, None]
        return x.transpose(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :length]

    def attend(self, table, lens, cu, q, scale, window=0):
        """q [T, Hq, d] -> o [T, Hq, d], lse [T, Hq] in float64; rows outside every sequence are NaN."""
        q = np.asarray(q, dtype=np.float64)
        o, lse = np.full(q.shape, np.nan), np.full(q.shape[:2], np.nan)
        H = self.codes["k"].shape[1]
        G = q.shape[1] // H
        for b, length in enumerate(lens):
            n = cu[b + 1] - cu[b]
            if n == 0:
                continue
            k, v = self.read("k", table[b], length), self.read("v", table[b], length)
            for i in range(n):
                r, p = cu[b] + i, length - n + i
                lo = max(p - window + 1, 0) if window else 0
                if p < lo:
                    o[r], lse[r] = 0.0, -np.inf
                    continue
                for h in range(q.shape[1]):
                    s = scale * (k[h // G, lo:p + 1] @ q[r, h])
                    m = s.max()
                    w = np.exp(s - m)
                    o[r, h] = (w @ v[h // G, lo:p + 1]) / w.sum()
                    lse[r, h] = m + math.log(w.sum())
        return o, lse
