"""Inputs for the tests of the 4-bit key/value cache: ragged batches over shuffled pages, caches
filled with random bytes, and the tolerance of the attention."""
from __future__ import annotations

import numpy as np

from oracle import kv4_oracle as K


def page_bytes(H, D, page, G):
    return H * page * (D + 4 * D // G)


def batch(rows, lens, page, extra_pages=2, extra_rows=0, seed=0):
    """cu int32 [B + 1], lens int32 [B], table int32 [B, max_pages], pages, T."""
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    per = [-(-n // page) for n in lens]
    width = max(max(per), 1)
    pages = sum(per) + extra_pages
    order = rng.permutation(pages)
    table = np.full((len(lens), width), 2 ** 30, dtype=np.int32)  # never looked up
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    return cu, np.array(lens, dtype=np.int32), table, pages, int(cu[-1]) + extra_rows


def random_cache(pages, H, D, page, G, fmt, held=None, seed=0, low=-3.0, high=-1.0):
    """A cache of random codes with scales 2^[low, high).  held: set of (page, slot); every
    scale elsewhere is a NaN or an infinity, which must not matter."""
    rng = np.random.default_rng(seed + 1000)
    data = rng.integers(0, 256, (pages, page_bytes(H, D, page, G)), dtype=np.uint8)
    c = K.Cache(data, H, D, page, G)
    n = D // G
    bits = np.float32(2.0 ** rng.uniform(low, high, (pages, H, page, 2, n))).view(np.uint32) >> 16
    junk = rng.choice([0x7FC0, 0x7F80, 0xFF80, 0xFFFF], (pages, H, page, 2, n))
    if held is not None:
        mask = np.zeros((pages, page), dtype=bool)
        for p, s in held:
            mask[p, s] = True
        bits = np.where(mask[:, None, :, None, None], bits, junk)
    for h in range(H):
        for s in range(page):
            _, ks, _, vs = c._off(h, s)
            for g in range(n):
                for at, j in ((ks + 2 * g, 0), (vs + 16 * g, 1)):
                    data[:, at] = bits[:, h, s, j, g] & 255
                    data[:, at + 1] = bits[:, h, s, j, g] >> 8
    return c


def held_of(lens, table, page):
    return {(int(table[b, p // page]), p % page) for b in range(len(lens)) for p in range(lens[b])}


def bf16_bits(x):
    """bf16 patterns (uint16) of float32 values, nearest even."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def attention_bounds(want, slack, D):
    """Largest difference that the arithmetic allows, for outputs and for lse.

    A score is a sum of D exact products in fp32 (error at most D 2^-24 sum |q k|), then one
    multiplication, one subtraction and an exponential with an error of an ulp: relative to the
    exponential's argument, at most d = (D + 4) 2^-24 qk + 4 * 2^-24 (1 + |argument|), where the
    argument is at most 2 qk + 8 / log2(e).  Each weight is rounded to fp16 (2^-11 of itself, or
    2^-25 absolute where it is subnormal, against a largest weight of 2^4), the sums of n terms
    are fp32, and the result is rounded to bf16 (2^-8 of itself)."""
    out, _ = want
    pv, qk, seen, vmax = slack
    d = (D + 4) * 2.0 ** -24 * qk + 4 * 2.0 ** -24 * (1 + 2 * qk + 6)
    rel = 2.0 ** -11 + 2 * np.expm1(d) + 2 * (seen + 8) * 2.0 ** -24
    bound = (2.0 ** -8 * np.abs(out) + rel[..., None] * pv * (1 + 2.0 ** -8)
             + (2.0 ** -29 * seen * vmax)[..., None] + 2.0 ** -130)
    lse_bound = d + (seen + 8) * 2.0 ** -24 + 4 * 2.0 ** -24 * (np.abs(want[1]) + 1)
    return bound, lse_bound
