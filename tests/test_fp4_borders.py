"""Why the 4-bit append's arithmetic gives the codes of exact quotients: every quotient that its format allows
either lies on a rounding border exactly or keeps a distance from it that the arithmetic's errors do not bridge."""

from fractions import Fraction

BORDERS = [Fraction(n, 4) for n in (1, 3, 5, 7, 10, 14, 20)]       # halfway between neighbouring e2m1 magnitudes


def test_quotients_by_a_scale():
    """x of 8 bits over s of up to 4 (e4m3, subnormal ones among them): within one part in 2^9 of a border only on it.
    The kernel's quotient is off by 2^-11 (fp16) and 2^-22 (a product with a reciprocal)."""
    near = 0
    for x in range(128, 256):
        for s in [*range(8, 16), *range(1, 8)]:
            for e in range(-14, 8):
                q = Fraction(x, s) * Fraction(2) ** e
                for b in BORDERS:
                    off = abs(q / b - 1)
                    assert off == 0 or off > Fraction(1, 1 << 9)
                    near += off == 0
    assert near > 0


def test_scales():
    """A block's largest magnitude (8 bits) over 6: the product with fl(1 / 6), which is off by 2^-25 and
    rounded once more (2^-24), against the borders between e4m3 numbers (odd 5-bit numbers, and below 2^-6 odd
    multiples of 2^-10)."""
    sixth = Fraction(float.fromhex("0x1.555556p-3"))
    assert abs(sixth * 6 - 1) == Fraction(1, 1 << 25)
    ties = 0
    for m in range(128, 256):
        for e in range(-12, 10):
            exact = Fraction(m, 128) * Fraction(2) ** e / 6
            step = Fraction(1, 1 << 9)
            while exact >= 16 * step:
                step *= 2
            r = exact / step - Fraction(1, 2)                          # whole where halfway
            if r.denominator == 1:
                ties += 1
                got = Fraction(m, 128) * Fraction(2) ** e * sixth      # rounded to 24 bits this is the border itself
                ulp = Fraction(1, 1 << 24)
                while exact >= (1 << 24) * ulp:
                    ulp *= 2
                while exact < (1 << 23) * ulp:
                    ulp /= 2
                assert abs(got - exact) < ulp / 2 and (exact / ulp).denominator == 1
            else:
                off = abs(r - round(r)) * step / exact
                assert off > Fraction(1, 1 << 20)
    assert ties > 0
