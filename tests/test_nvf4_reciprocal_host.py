"""The quotients of the NVF4 quantizer (csrc/nvf4_quant.cu) where its row scales are powers of
two: products by an FP32 reciprocal that find every value in the middle between two codes, in
exact arithmetic."""

from fractions import Fraction

MIDDLES = [Fraction(n, 4) for n in (1, 3, 5, 7, 10, 14, 20)]  # between E2M1's magnitudes


def fp32(x, mode):
    """x > 0 with 24 significant bits, rounded "up", to "zero" or to "nearest" (ties to even)."""
    e = 0
    while Fraction(2) ** e > x:
        e -= 1
    while Fraction(2) ** (e + 1) <= x:
        e += 1
    step = Fraction(2) ** (e - 23)
    n, rest = divmod(x, step)
    rest /= step
    if (mode == "up" and rest) or (mode == "nearest" and (rest, n % 2) > (Fraction(1, 2), 0)):
        n += 1
    return n * step


def missed(reciprocal, product):
    return sum(fp32(m * d * fp32(Fraction(1, d), reciprocal), product) != m
               for d in range(1, 16) for m in MIDDLES)  # an E4M3 scale has 4 significant bits


def test_rounding():
    third = Fraction(1, 3)
    assert fp32(third, "zero") < third < fp32(third, "up")
    assert fp32(Fraction(2 ** 24 + 1), "nearest") == 2 ** 24
    assert fp32(Fraction(2 ** 24 + 3), "nearest") == 2 ** 24 + 4
    assert fp32(Fraction(5, 8), "up") == Fraction(5, 8)


def test_codes():
    assert missed("up", "zero") == 0
    assert missed("nearest", "nearest") == missed("up", "nearest") == 14


def test_scales():
    # largest values whose sixth is in the middle between two E4M3 codes (5 significant bits)
    sixth = fp32(Fraction(1, 6), "nearest")
    assert all(fp32(6 * t * sixth, "nearest") == t for t in range(16, 32))
