"""CPU oracle of the paged 4-bit key/value cache, in 64 bits and with plain loops.

Written from the format (include/trellis_kv4.h states it) and sharing no code with the GPU
path: a head's vector in blocks of 128, each rotated with the normalised Sylvester
Hadamard, one bf16 scale (largest magnitude / 6) and E2M1 codes, nearest with ties to even.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MIDPOINTS = (MAGNITUDES[1:] + MAGNITUDES[:-1]) / 2


def hadamard128() -> np.ndarray:
    h = np.ones((1, 1))
    while h.shape[0] < 128:
        h = np.block([[h, h], [h, -h]])
    return h / math.sqrt(128.0)


H = hadamard128()


def bf16_bits(x: np.ndarray) -> np.ndarray:
    """Nearest bf16 (ties to even) of finite float64 values, as bit patterns: by float32 first
    rounded to odd, so the two roundings are one."""
    x = np.asarray(x, np.float64)
    f = x.astype(np.float32)
    bits = f.view(np.uint32).astype(np.int64)
    err = x - f.astype(np.float64)
    # round to odd: truncate towards zero, then set the last bit where anything was lost
    away = (np.abs(f.astype(np.float64)) > np.abs(x))
    bits = np.where(away, bits - 1, bits)
    bits = np.where(err != 0, bits | 1, bits)
    low, up = bits & 0xFFFF, bits >> 16
    up = up + ((low > 0x8000) | ((low == 0x8000) & (up & 1 == 1)))
    return up.astype(np.uint16)


def bf16_value(bits: np.ndarray) -> np.ndarray:
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def e2m1_codes(y: np.ndarray) -> np.ndarray:
    """Nearest E2M1 code, ties to the even code, magnitudes over 6 become 6; bit 3 the sign."""
    a = np.abs(y)
    c = np.searchsorted(MIDPOINTS, a, side="left")  # a midpoint goes to the lower code ...
    c = c + (np.isin(a, MIDPOINTS) & (c % 2 == 1))  # ... or to the upper, where that is even
    return (c | np.where(np.signbit(y), 8, 0)).astype(np.uint8)


def e2m1_values(codes: np.ndarray) -> np.ndarray:
    c = np.asarray(codes)
    return np.where(c & 8, -1.0, 1.0) * MAGNITUDES[c & 7]


def quantize(x: np.ndarray):
    """x [..., 128] -> (codes uint8 [..., 128], scale bits uint16 [...])."""
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x).all(-1)
    r = np.where(bad[..., None], 0.0, x) @ H
    s = bf16_bits(np.abs(r).max(-1) / 6.0)
    sv = bf16_value(s)
    small = sv < 2.0 ** -126
    s = np.where(small, 0, s).astype(np.uint16)
    codes = e2m1_codes(r / np.where(small, 1.0, sv)[..., None])
    codes = np.where((small | bad)[..., None], 0, codes).astype(np.uint8)
    return codes, np.where(bad, 0x7FC0, s).astype(np.uint16)


class Cache:
    """The pool [n_layers][n_pages][n_kv_heads][chunk] as numpy bytes, and its operations."""

    def __init__(self, n_layers: int, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int,
                 pool: Optional[np.ndarray] = None):
        self.L, self.P, self.T, self.Hk, self.D = n_layers, n_pages, page_size, n_kv_heads, head_dim
        self.NB = head_dim // 128
        chunk = 132 * self.NB * page_size
        self.pool = np.zeros((n_layers, n_pages, n_kv_heads, chunk), np.uint8) if pool is None else \
            pool.reshape(n_layers, n_pages, n_kv_heads, chunk)

    def at(self, which: int, nb: int, t: int):
        """(offset of the 64 code bytes, offset of the scale) of token t of a page."""
        part = which * self.NB + nb
        return (part * self.T + t) * 64, 128 * self.NB * self.T + (part * self.T + t) * 2

    def put(self, layer: int, page: int, t: int, k: np.ndarray, v: np.ndarray) -> None:
        """k, v [n_kv_heads, head_dim]: one token."""
        for which, x in ((0, k), (1, v)):
            codes, s = quantize(np.asarray(x, np.float64).reshape(self.Hk, self.NB, 128))
            for nb in range(self.NB):
                c, a = self.at(which, nb, t)
                self.pool[layer, page, :, c:c + 64] = codes[:, nb, ::2] | (codes[:, nb, 1::2] << 4)
                self.pool[layer, page, :, a:a + 2] = s[:, nb, None].view(np.uint8)

    def parts(self, layer: int, page: int, t: int, which: int):
        """(codes [n_kv_heads, NB, 128], scale bits [n_kv_heads, NB]) of one token."""
        codes = np.zeros((self.Hk, self.NB, 128), np.uint8)
        s = np.zeros((self.Hk, self.NB), np.uint16)
        for nb in range(self.NB):
            c, a = self.at(which, nb, t)
            b = self.pool[layer, page, :, c:c + 64]
            codes[:, nb, ::2], codes[:, nb, 1::2] = b & 15, b >> 4
            s[:, nb] = np.ascontiguousarray(self.pool[layer, page, :, a:a + 2]).view(np.uint16)[:, 0]
        return codes, s

    def rows(self, layer: int, row: Sequence[int], length: int, which: int) -> np.ndarray:
        """The keys (0) or values (1) of a sequence with the table row `row`, rotated back:
        [length, n_kv_heads, head_dim]."""
        out = np.zeros((length, self.Hk, self.NB, 128))
        for p in range(length):
            codes, s = self.parts(layer, int(row[p // self.T]), p % self.T, which)
            out[p] = e2m1_values(codes) * bf16_value(s)[..., None]
        return (out @ H).reshape(length, self.Hk, self.D)


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, window: int = 0, sinks: int = 0):
    """q [n, heads, D] (the last n tokens), k, v [length, kv heads, D] -> (y [n, heads, D],
    lse [n, heads], mass [n, heads, D] = sum_j p_j |v_j|, spread [n, heads] = the largest
    |scale| * sum_d |q_d k_d| over visible keys)."""
    q = np.asarray(q, np.float64)
    n, heads, D = q.shape
    length, hk = k.shape[0], k.shape[1]
    y, mass = np.zeros((n, heads, D)), np.zeros((n, heads, D))
    lse, spread = np.full((n, heads), -np.inf), np.zeros((n, heads))
    j = np.arange(length)
    for i in range(n):
        p = length - n + i
        see = j <= p
        if window:
            see &= (j > p - window) | (j < sinks)
        if not see.any():
            continue
        for h in range(heads):
            kk, vv = k[see, h // (heads // hk)], v[see, h // (heads // hk)]
            s = scale * (kk @ q[i, h])
            m = s.max()
            e = np.exp(s - m)
            l = e.sum()
            y[i, h] = e @ vv / l
            mass[i, h] = e @ np.abs(vv) / l
            lse[i, h] = m + math.log(l) if np.isfinite(m) else m + l
            spread[i, h] = abs(scale) * np.abs(kk * q[i, h]).sum(-1).max()
    return y, lse, mass, spread


class Pages:
    """Tables, lengths and counts, and the page operations, one item at a time."""

    def __init__(self, cache: Cache, table: np.ndarray, lens: np.ndarray, ref: np.ndarray):
        self.c, self.table, self.lens, self.ref = cache, table, lens, ref

    def _n(self, length: int) -> int:
        return -(-int(length) // self.c.T)

    def _take(self, need: int):
        free = [g for g in range(self.c.P) if self.ref[g] == 0]
        return free[:need] if len(free) >= need else None

    def _drop(self, slot: int) -> None:
        for j in range(self._n(self.lens[slot])):
            self.ref[self.table[slot, j]] -= 1
        self.lens[slot] = 0

    def reserve(self, slots, add) -> bool:
        need = [self._n(self.lens[s] + a) - self._n(self.lens[s]) for s, a in zip(slots, add)]
        pages = self._take(sum(need))
        if pages is None:
            return False
        for s, a, n in zip(slots, add, need):
            h = self._n(self.lens[s])
            for j in range(n):
                g = pages.pop(0)
                self.table[s, h + j], self.ref[g] = g, 1
            self.lens[s] += a
        return True

    def fork(self, src, dst) -> bool:
        pages = self._take(sum(int(self.lens[s]) % self.c.T != 0 for s in src))
        if pages is None:
            return False
        for s, d in zip(src, dst):
            self._drop(d)
            full, part = divmod(int(self.lens[s]), self.c.T)
            for j in range(full):
                self.table[d, j] = self.table[s, j]
                self.ref[self.table[s, j]] += 1
            if part:
                g, a = pages.pop(0), self.table[s, full]
                self.table[d, full], self.ref[g] = g, 1
                for t in range(part):
                    self._copy(a, t, g, t)
            self.lens[d] = self.lens[s]
        return True

    def _copy(self, a: int, t: int, g: int, u: int) -> None:
        p = self.c.pool
        for which in (0, 1):
            for nb in range(self.c.NB):
                (c0, s0), (c1, s1) = self.c.at(which, nb, t), self.c.at(which, nb, u)
                p[:, g, :, c1:c1 + 64] = p[:, a, :, c0:c0 + 64]
                p[:, g, :, s1:s1 + 2] = p[:, a, :, s0:s0 + 2]

    def compact(self, src, dst, keeps) -> bool:
        need = [self._n(len(k)) for k in keeps]
        pages = self._take(sum(need))
        if pages is None:
            return False
        new = []
        for s, k, n in zip(src, keeps, need):
            mine = [pages.pop(0) for _ in range(n)]
            for u, pos in enumerate(k):
                self._copy(self.table[s, pos // self.c.T], pos % self.c.T, mine[u // self.c.T], u % self.c.T)
            new.append(mine)
        for d, k, mine in zip(dst, keeps, new):
            self._drop(d)
            for j, g in enumerate(mine):
                self.table[d, j], self.ref[g] = g, 1
            self.lens[d] = len(k)
        return True

    def free(self, slots) -> None:
        for s in slots:
            self._drop(s)
