"""Quotients of the slot appends' quantisers, by whole-number arithmetic: with y the rounded reciprocal of s and q = x y rounded,
q - (q s - x) y is the rounded quotient x / s for every scale that the append forms (s = absmax / 6 or / 448, rounded) and every
bf16 x up to absmax, so that one correction is enough there; for any s two are needed. The same for these scales themselves."""
import pytest


def rn(num, den):
    """num / den (positive) rounded to 24 bits, ties to even, as (mantissa, exponent)."""
    e = num.bit_length() - den.bit_length() - 24
    while True:
        n, d = (num, den << e) if e >= 0 else (num << -e, den)
        m, r = divmod(n, d)
        if m >= 1 << 24:
            e += 1
            continue
        if m < 1 << 23:
            e -= 1
            continue
        m += 2 * r > d or (2 * r == d and m & 1)
        return (m, e) if m < 1 << 24 else (m >> 1, e + 1)


def rounded(num, exponent):
    """num * 2^exponent rounded to 24 bits, as (signed mantissa, exponent)."""
    if num == 0:
        return 0, 0
    m, e = rn(abs(num), 1)
    return (m if num > 0 else -m), e + exponent


def fma(a, b, c):
    """a b + c, rounded once; operands and result (mantissa, exponent)."""
    n, e = a[0] * b[0], a[1] + b[1]
    low = min(e, c[1])
    return rounded((n << (e - low)) + (c[0] << (c[1] - low)), low)


@pytest.mark.parametrize("most,steps", [(6, 8), (448, 21)])
def test_one_correction_gives_the_rounded_quotient(most, steps):
    for a in range(128, 256):
        s = rn(a, most)
        y = rn(1 << 60, s[0])
        y = (y[0], y[1] - 60 - s[1])
        for j in range(steps):  # powers of two down to where every code is 0
            for x in range(128, a + 1 if j == 0 else 256):
                value = (x, -j)
                q = fma(value, y, (0, 0))
                left = fma(s, q, (-value[0], value[1]))
                q = fma((-left[0], left[1]), y, q)
                want = rn(x << 60, s[0])
                want = (want[0], want[1] - 60 - s[1] - j)
                assert q == want, (a, x, j)


@pytest.mark.parametrize("most", [6, 448])
def test_one_correction_gives_the_scale(most):
    """absmax / 6 and / 448 from their rounded reciprocals, for every bf16 mantissa."""
    y = rn(1, most)
    for a in range(128, 256):
        q = fma((a, 0), y, (0, 0))
        left = fma((-most, 0), q, (a, 0))
        assert fma(left, y, q) == rn(a, most), a
