"""CPU pins of the 4-bit cache's oracle: hand-worked codes and bytes, exact ties, an identity, and a
brute-force attention."""
import math
from fractions import Fraction

import numpy as np
import pytest

import kv4_util as U
from oracle import kv4_oracle as K


def test_grids():
    assert K.grid(K.FMT_INT4) == [float(v) for v in range(-8, 8)]
    assert K.grid(K.FMT_FP4) == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]


def test_encode_by_hand():
    # scale 1: amax 7 (INT4), 6 (FP4); ties go to the even code
    x = np.array([7, 0.5, 1.5, 2.5, -0.5, -1.5, -7, 0.0], dtype=float)
    codes, bits = K.encode_group(x, K.FMT_INT4)
    assert bits == 0x3F80 and codes == [15, 8, 10, 10, 8, 6, 1, 8]
    x = np.array([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -5, 0.0], dtype=float)
    codes, bits = K.encode_group(x, K.FMT_FP4)
    assert bits == 0x3F80 and codes == [7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 14, 0]
    for fmt, zero in ((K.FMT_INT4, 8), (K.FMT_FP4, 0)):
        assert K.encode_group(np.array([0.0, -0.0]), fmt) == ([zero, 8], 0)  # FP4 keeps signs
        assert K.encode_group(np.array([2.0 ** -101]), fmt) == ([zero], 0)
        assert K.encode_group(np.array([math.inf, 1]), fmt)[1] == 0x7FC0
        assert K.encode_group(np.array([math.nan]), fmt)[1] == 0x7FC0


@pytest.mark.parametrize("div", [6, 7])
def test_scales_are_never_near_a_rounding_tie(div):
    """a / 6 and a / 7 of every bf16 mantissa a lie at least 2^-12 of themselves away from a
    midpoint of two bf16 values, so rounding a float64 or float32 quotient is exact."""
    for a in range(128, 256):
        q = Fraction(a, div)
        e = math.floor(math.log2(q)) - 7
        pos = q / Fraction(2) ** e
        frac = pos - math.floor(pos)
        assert abs(frac - Fraction(1, 2)) / pos > Fraction(1, 4096), a


@pytest.mark.parametrize("fmt", [K.FMT_INT4, K.FMT_FP4])
def test_quotients_are_ties_or_far_from_them(fmt):
    """x / s of two 8-bit mantissas is a midpoint of the grid or at least 1 / 1020 away from every
    one: rounding the quotient to multiples of 2^-13 first cannot change a code."""
    g = sorted(set(K.grid(fmt)))
    mids = [Fraction(a + b) / 2 for a, b in zip(g, g[1:]) if a >= 0]
    for m in mids:
        for b in range(128, 256):
            for e in range(-6, 5):
                a0 = m * b / Fraction(2) ** e
                for a in (math.floor(a0), math.floor(a0) + 1):
                    if 128 <= a < 256:
                        y = Fraction(a, b) * Fraction(2) ** e
                        assert y == m or abs(y - m) >= Fraction(1, 1020)


def test_bytes_by_hand():
    """One head, D = 64, G = 32, a page of 32: where each nibble and scale lies."""
    data = np.zeros((1, U.page_bytes(1, 64, 32, 32)), dtype=np.uint8)
    c = K.Cache(data, 1, 64, 32, 32)
    k, v = np.zeros(64), np.zeros(64)
    k[0], k[33], v[2], v[63] = 7.0, -7.0, 14.0, -7.0
    c.put(0, 0, 13, k, v, K.FMT_INT4)
    row = data[0]
    assert row[13 * 32] == 0x8F            # d 0 low nibble 15, d 1 high nibble 8
    assert row[13 * 32 + 16] == 0x18       # d 32 = 0, d 33 = -7
    ks = 32 * 32
    assert list(row[ks + 13 * 4: ks + 13 * 4 + 4]) == [0x80, 0x3F, 0x80, 0x3F]
    vc = ks + 32 * 4
    assert row[vc + 64 * 4 + 2 * 4 + 2] == 0xF0   # block 1, d 2, positions 12 | 13
    assert row[vc + 64 * 4 + 63 * 4 + 2] == 0x10
    vs = vc + 32 * 32
    at = vs + 2 * (1 * 2 * 8 + 5)                  # block 1, group 0, position 5 of the block
    assert list(row[at:at + 2]) == [0x00, 0x40]    # 14 / 7 = 2
    kk, vv = c.get(0, 0, 13, K.FMT_INT4)
    assert np.array_equal(kk, k) and np.array_equal(vv, v)


@pytest.mark.parametrize("fmt", [K.FMT_INT4, K.FMT_FP4])
def test_grid_values_survive(fmt):
    """Rows of grid values times a power of two come back exactly."""
    rng = np.random.default_rng(1)
    cu, lens, table, pages, T = U.batch([5, 0, 9], [40, 7, 9], 32)
    vals = [x for x in K.grid(fmt) if abs(x) < 8]
    top = max(vals)
    k = rng.choice(vals, (T, 2, 64)) * 0.25
    k[..., ::32] = top * 0.25
    v = rng.choice(vals, (T, 2, 64)) * 4
    v[..., 1::32] = top * 4
    c = U.random_cache(pages, 2, 64, 32, 32, fmt)
    K.write(c, k, v, cu, lens, table, fmt)
    k2, v2 = K.read(c, T, cu, lens, table, fmt)
    assert np.array_equal(k, k2) and np.array_equal(v, v2)


def test_attention_against_exact_sums():
    """Against exponentials summed in Fractions of 60-digit decimals, with a window and sinks."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    fmt, page = K.FMT_FP4, 32
    cu, lens, table, pages, T = U.batch([3, 1], [37, 0], page)
    c = U.random_cache(pages, 1, 64, page, 32, fmt, held=U.held_of(lens, table, page))
    q = U.K.bf16_value(U.bf16_bits(np.random.default_rng(3).normal(size=(T, 2, 64))))
    out, lse, _ = K.attention(c, q, cu, lens, table, fmt, 0.125, window=9, sinks=2)
    assert np.array_equal(out[3], np.zeros((2, 64))) and np.all(np.isneginf(lse[3]))
    for i in range(3):
        p = 34 + i
        seen = [t for t in range(p + 1) if t > p - 9 or t < 2]
        assert len(seen) == 11
        kv = [c.get(int(table[0, t // page]), 0, t % page, fmt) for t in seen]
        for h in range(2):
            e = [sum((Decimal(float(a)) * Decimal(float(b)) for a, b in zip(k, q[i, h])),
                     Decimal(0)) / 8 for k, _ in kv]
            w = [x.exp() for x in e]
            tot = sum(w)
            assert abs(float(tot.ln()) - lse[i, h]) < 1e-13 * max(1, abs(lse[i, h]))
            for d in range(0, 64, 7):
                want = sum(a * Decimal(float(v[d])) for a, (_, v) in zip(w, kv)) / tot
                assert abs(float(want) - out[i, h, d]) < 1e-13
