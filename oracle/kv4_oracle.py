"""CPU oracle for the 4-bit key/value cache: writing, reading back and attention.

TEST INFRASTRUCTURE ONLY, like ``moe_oracle``: float64 (and exact comparisons of bf16 values),
one row, head and group at a time, no code shared with the HIP library.

Cache layout (uint8 [pages, bytes]): a page holds, for each kv head in turn,
``page`` positions as K codes [page, D/2] (byte i: d = 2i low nibble, 2i+1 high), K scales
[page, D/G] bf16, V codes [page/8, D, 4] (byte i of a block and d: position 2i low, 2i+1 high) and
V scales [page/8, D/G, 8] bf16.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

FMT_INT4, FMT_FP4 = 0, 1
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def grid(fmt):
    """Value of each of the 16 codes."""
    if fmt == FMT_INT4:
        return [float(c - 8) for c in range(16)]
    return list(E2M1) + [-e for e in E2M1]


def bf16_bits(x: float) -> int:
    """Nearest bf16 of a positive float64 in bf16's normal range (ties to even), as 16 bits."""
    m, e = math.frexp(x)
    rounded = math.ldexp(round(Fraction(m) * 256), e - 8)
    return int(np.float32(rounded).view(np.uint32)) >> 16


def bf16_value(bits) -> np.ndarray:
    b = np.asarray(bits, dtype=np.uint32) << 16
    return b.view(np.float32).astype(np.float64)


def encode_group(x: np.ndarray, fmt: int):
    """(codes, scale bits) of one group of values (float64, each a bf16 value)."""
    if not np.all(np.isfinite(x)):
        return None, 0x7FC0
    top = float(np.max(np.abs(x)))
    if top < 2.0 ** -100:
        return [8 if fmt == FMT_INT4 or math.copysign(1.0, v) < 0 else 0 for v in x], 0
    # (the float64 quotient is no bf16 tie and none is near: see the pins)
    bits = bf16_bits(top / (7 if fmt == FMT_INT4 else 6))
    scale = Fraction(float(bf16_value(bits)))
    codes = []
    for v in x:
        y = Fraction(float(v)) / scale
        if fmt == FMT_INT4:
            codes.append(min(max(round(y), -8), 7) + 8)  # round(): ties to even
        else:
            m = abs(y)
            best = 0
            for c in range(1, 8):
                mid = (Fraction(E2M1[c - 1]) + Fraction(E2M1[c])) / 2
                if m > mid or (m == mid and c % 2 == 0):
                    best = c
            codes.append(best + (8 if math.copysign(1.0, v) < 0 else 0))
    return codes, bits


class Cache:
    """Byte addressing of one cache."""

    def __init__(self, data: np.ndarray, kv_heads: int, dim: int, page: int, group: int):
        self.data, self.H, self.D, self.page, self.G = data, kv_heads, dim, page, group
        self.head_bytes = page * (dim + 4 * dim // group)
        assert data.shape[1] == kv_heads * self.head_bytes

    def _off(self, head, slot):
        n = self.D // self.G
        base = head * self.head_bytes
        kc = base + slot * self.D // 2
        ks = base + self.page * self.D // 2 + 2 * slot * n
        v0 = base + self.page * self.D // 2 + 2 * self.page * n
        vc = v0 + (slot // 8) * self.D * 4 + (slot % 8) // 2
        vs = v0 + self.page * self.D // 2 + 2 * ((slot // 8) * n * 8 + slot % 8)
        return kc, ks, vc, vs

    def _put_scale(self, page, at, bits):
        self.data[page, at] = bits & 255
        self.data[page, at + 1] = bits >> 8

    def _scale(self, page, at):
        return float(bf16_value(int(self.data[page, at]) | int(self.data[page, at + 1]) << 8))

    def put(self, page, head, slot, k, v, fmt):
        """Stores one row; codes of a group that is not finite are unspecified (left alone)."""
        kc, ks, vc, vs = self._off(head, slot)
        row = self.data[page]
        for g in range(self.D // self.G):
            codes, bits = encode_group(k[g * self.G:(g + 1) * self.G], fmt)
            self._put_scale(page, ks + 2 * g, bits)
            for i, c in enumerate(codes or []):
                d = g * self.G + i
                at, sh = kc + d // 2, 4 * (d % 2)
                row[at] = (int(row[at]) & ~(15 << sh) & 255) | c << sh
            codes, bits = encode_group(v[g * self.G:(g + 1) * self.G], fmt)
            self._put_scale(page, vs + 16 * g, bits)
            for i, c in enumerate(codes or []):
                at, sh = vc + 4 * (g * self.G + i), 4 * (slot % 2)
                row[at] = (int(row[at]) & ~(15 << sh) & 255) | c << sh

    def get(self, page, head, slot, fmt):
        """(k, v) of one position, float64 [D]."""
        kc, ks, vc, vs = self._off(head, slot)
        row, val = self.data[page], grid(fmt)
        n = self.D // self.G
        d = np.arange(self.D)
        lut = np.array(val)
        k = lut[(row[kc + d // 2] >> (4 * (d % 2))) & 15]
        v = lut[(row[vc + 4 * d] >> (4 * (slot % 2))) & 15]
        sk = np.repeat([self._scale(page, ks + 2 * g) for g in range(n)], self.G)
        sv = np.repeat([self._scale(page, vs + 16 * g) for g in range(n)], self.G)
        with np.errstate(invalid="ignore"):
            return k * sk, v * sv


def _page_of(cache, table, b, p):
    """Page of position p of sequence b, or None where it has none."""
    if p < 0 or p >= table.shape[1] * cache.page:
        return None
    page = int(table[b, p // cache.page])
    return page if 0 <= page < cache.data.shape[0] else None


def rows_of(cu, lens):
    """(row, sequence, position) of every row."""
    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        for i in range(n):
            yield int(cu[b]) + i, b, int(lens[b]) - n + i


def write(cache: Cache, k, v, cu, lens, table, fmt):
    """k, v float64 [T, H, D]; changes cache.data."""
    for t, b, p in rows_of(cu, lens):
        page = _page_of(cache, table, b, p)
        if page is None:
            continue
        for h in range(cache.H):
            cache.put(page, h, p % cache.page, k[t, h], v[t, h], fmt)


def read(cache: Cache, T, cu, lens, table, fmt):
    """(k, v) float64 [T, H, D]; rows of nobody are NaN, rows without a place are zero."""
    k = np.full((T, cache.H, cache.D), np.nan)
    v = np.full((T, cache.H, cache.D), np.nan)
    for t, b, p in rows_of(cu, lens):
        page = _page_of(cache, table, b, p)
        for h in range(cache.H):
            if page is None:
                k[t, h], v[t, h] = 0.0, 0.0
            else:
                k[t, h], v[t, h] = cache.get(page, h, p % cache.page, fmt)
    return k, v


def attention(cache: Cache, q, cu, lens, table, fmt, scale, window=0, sinks=0):
    """(out, lse, slack): out float64 [T, Hq, D], lse [T, Hq], and per row and head what an error
    bound needs: sum p |v| [T, Hq, D], the largest sum |q k| |scale| over visible positions
    [T, Hq], the number of visible positions [T, Hq] and the largest |v| [T, Hq]."""
    T, Hq, D = q.shape
    r = Hq // cache.H
    out = np.full((T, Hq, D), np.nan)
    lse = np.full((T, Hq), np.nan)
    pv = np.zeros((T, Hq, D))
    qk = np.zeros((T, Hq))
    seen = np.zeros((T, Hq))
    vmax = np.zeros((T, Hq))
    held = {}
    for t, b, p in rows_of(cu, lens):
        pos = [s for s in range(0, p + 1)
               if (window == 0 or s > p - window or s < sinks) and
               _page_of(cache, table, b, s) is not None]
        for kv in range(cache.H):
            if (b, kv) not in held:
                held[b, kv] = {}
            for s in pos:
                if s not in held[b, kv]:
                    held[b, kv][s] = cache.get(_page_of(cache, table, b, s), kv, s % cache.page, fmt)
            k = np.array([held[b, kv][s][0] for s in pos]).reshape(len(pos), D)
            v = np.array([held[b, kv][s][1] for s in pos]).reshape(len(pos), D)
            for h in range(kv * r, (kv + 1) * r):
                if not pos:
                    out[t, h], lse[t, h] = 0.0, -math.inf
                    continue
                x = (k @ q[t, h]) * scale
                m = np.max(x)
                e = np.exp(x - m)
                out[t, h] = (e @ v) / e.sum()
                lse[t, h] = m + math.log(e.sum())
                pv[t, h] = (e @ np.abs(v)) / e.sum()
                qk[t, h] = np.max(np.abs(k) @ np.abs(q[t, h])) * abs(scale)
                seen[t, h] = len(pos)
                vmax[t, h] = np.max(np.abs(v))
    return out, lse, (pv, qk, seen, vmax)
