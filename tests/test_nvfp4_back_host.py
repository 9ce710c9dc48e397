"""The read-back's quotient on the host (no GPU): decode(sf) / gs by Markstein's
correction of a product with the correctly rounded reciprocal,

  inv = RN(1 / gs),  q = RN(d inv),  e = RN(d - q gs),  r = RN(q + e inv)

is RN(d / gs) for every significand of gs and every significand that an E4M3 code
has.  Powers of two change no rounding while nothing under- or overflows: with
2^-9 <= d <= 448 and 2^-100 < gs < 2^100, e is a multiple of 2^-47 d or zero, and
the others lie within 2^+-110."""
import numpy as np

F = np.float32


def fma(a, b, c):
    """RN(a b + c) of float32: the product is exact in float64, the sum is rounded
    to odd there (53 >= 24 + 2 bits), so the second rounding is the only one."""
    p, c = a.astype(np.float64) * b, c.astype(np.float64)
    s = p + c
    t = s - p
    err = (p - (s - t)) + (c - t)
    fix = (err != 0) & (s.view(np.int64) % 2 == 0)
    s[fix] = np.nextafter(s[fix], np.where(err[fix] > 0, np.inf, -np.inf))
    return s.astype(F)


def quotient(d, gs):
    """(by the correction, the product alone)"""
    inv = F(1) / gs
    q = d * inv
    return fma(fma(-q, gs, d), inv, q), q


def test_fma_rounds_once():
    one, tiny = F(1), F(2.0 ** -24)
    a = np.array([1 + 2 ** -12, 1 + 2 ** -12], F)
    b = np.array([1 + 2 ** -12, 1 - 2 ** -12], F)
    got = fma(a, b, np.array([tiny ** 2, -one], F))
    assert got[0] == F(1 + 2 ** -11 + 2 ** -23)  # 2^-24 + 2^-48 above the tie: up
    assert got[1] == F(-(2.0 ** -24))


def test_every_significand():
    wrong = 0
    for at in range(0, 1 << 23, 1 << 20):
        gs = (np.arange(at, at + (1 << 20), dtype=np.uint32) + 0x3F800000).view(F)
        for m in range(8):
            d = np.full_like(gs, 1 + m / 8)
            r, q = quotient(d, gs)
            want = d / gs
            assert np.array_equal(r, want), m
            wrong += int((q != want).sum())
    assert wrong > 1 << 20  # the product alone is off in many
