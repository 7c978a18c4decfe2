"""The 4-bit oracle against brute force and closed forms, and mistakes planted in
it that the pins find."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import fp8_ref, nvf4_ref as ref


def nearest(x):
    """Code of x by exact distances to the 8 magnitudes, ties to the even code."""
    mag = min(abs(Fraction(float(x))), Fraction(6))
    best = min(range(8), key=lambda c: (abs(mag - Fraction(float(ref.GRID[c]))), c % 2))
    return best | (8 if np.signbit(x) else 0)


def test_codes_are_the_nearest():
    x = np.concatenate([np.arange(-8, 8.01, 1 / 64), [0.0, -0.0, 1e-30, -1e-30, 1e30, np.inf]])
    x = np.concatenate([x, np.nextafter(x, 9), np.nextafter(x, -9)])
    assert [int(c) for c in ref.e2m1_codes(x)] == [nearest(min(v, 1e6)) for v in x]


@pytest.mark.parametrize("amax,r", [(2688.0, 1.0), (np.nextafter(2688.0, 3000), 2.0), (1344.0, 0.5),
                                    (0.0, 2.0 ** -100), (2688.0 * 2.0 ** -100, 2.0 ** -100),
                                    (65504.0, 32.0), (1.0, 2.0 ** -11)])
def test_row_scale(amax, r):
    assert ref.row_scale(amax) == r


def test_quantize_known_rows():
    # a block's largest value is 6 times its scale; blocks of exact codes come back exactly
    x = np.zeros((3, 40))
    x[0, :16] = np.tile([0, .5, 1, 1.5, 2, 3, 4, 6], 2) * np.where(np.arange(16) % 3, 1, -1) * 448
    x[0, 16:32] = x[0, :16] / 448 * 2.0 ** -9
    x[1, 35] = -3.0
    codes, scales, rows = ref.quantize(x)
    assert rows[0] == 1.0 and list(scales[0]) == [0x7E, 0x01, 0x01]
    assert np.array_equal(ref.values(codes, scales, rows)[0], x[0])
    assert rows[1] == 2.0 ** -9 and scales[1, 2] == fp8_ref.e4m3_codes(3.0 / 6 * 512)
    assert codes[1, 35] == 15 and (codes[1, :35] == 0).all()
    assert rows[2] == np.float32(2.0 ** -100) and (scales[2] == 1).all()


def test_quantize_error_and_special_values():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(6, 100)).astype(np.float32)
    x[1, 20], x[2, 99], x[3, 0] = np.inf, np.nan, -np.inf
    codes, scales, rows = ref.quantize(x)
    assert scales[1, 1] == scales[2, 6] == scales[3, 0] == ref.NAN
    assert (codes[1, 16:32] == 0).all() and np.count_nonzero(scales == ref.NAN) == 3
    v = ref.values(codes, scales, rows)
    ok = np.isfinite(v)
    # half the widest step (2 of 6) of the block's largest value, its scale rounded by 2^-4
    top = np.abs(np.nan_to_num(x, posinf=0.0, neginf=0.0))
    for j in range(7):
        at = np.s_[:, 16 * j:16 * (j + 1)]
        amax = top[at].max(1, keepdims=True)
        within = np.broadcast_to(amax / 6 * (1 + 2.0 ** -4), ok[at].shape)
        assert (np.abs(v[at] - x[at])[ok[at]] <= within[ok[at]]).all()
    given = np.array([1.0, 2.0 ** -101, 0.0, np.nan, -1.0, 2.0 ** -20])
    _, s, r = ref.quantize(np.ones((6, 16)), given)
    assert list(s[:, 0] == ref.NAN) == [False, True, True, True, True, False]
    assert ref.values(*ref.quantize(np.ones((6, 16)), given))[5, 0] == 6 * 448 * 2.0 ** -20


def test_pack_and_tiles():
    rng = np.random.default_rng(2)
    codes = rng.integers(0, 16, (5, 7)).astype(np.uint8)
    p = ref.pack(codes)
    assert p.shape == (5, 4) and (p[:, 3] < 16).all() and np.array_equal(ref.unpack(p, 7), codes)
    s = rng.integers(0, 127, (300, 9)).astype(np.uint8)
    t = ref.tiles(s)
    assert t.shape == (3, 3, 32, 16)
    # row 200 is row 72 of tile 1: line 8, third word; group 6 is byte 2 of tile column 1
    assert t[1, 1, 8, 8 + 2] == s[200, 6] and t[2, 2, 31, 3] == 0 and t.sum() == s.sum()


def test_product():
    rng = np.random.default_rng(3)
    a, b = rng.normal(size=(3, 20)), rng.normal(size=(4, 20))
    t, err = ref.product(a, b, alpha=0.5)
    want = [[float(sum(Fraction(x) * Fraction(y) for x, y in zip(u, v)) / 2) for v in b] for u in a]
    assert np.abs(t - want).max() < 1e-12 and (err > 0).all()


@pytest.mark.parametrize("mistake", ["ties", "grid", "floor", "group"])
def test_planted_mistakes_are_found(mistake, monkeypatch):
    if mistake == "ties":
        def codes(x):
            return np.minimum(np.searchsorted([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.], np.abs(x),
                                              side="right"), 7).astype(np.uint8) | (np.signbit(x) * 8)
        monkeypatch.setattr(ref, "e2m1_codes", codes)
        with pytest.raises(AssertionError):
            test_codes_are_the_nearest()
        return
    if mistake == "grid":
        monkeypatch.setattr(ref, "GRID", np.array([0, .5, 1, 1.5, 2, 3, 4, 5.]))
    elif mistake == "floor":
        monkeypatch.setattr(ref, "row_scale", lambda a: np.float32(2.0 ** np.floor(np.log2(
            max(a, 2.0 ** -80) / 2688))))
    else:
        monkeypatch.setattr(ref, "GROUP", 32)
    with pytest.raises((AssertionError, ValueError, IndexError)):
        test_quantize_known_rows()
