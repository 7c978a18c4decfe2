"""The 64-bit references of the FP8 and expert-routing operators, pinned by
hand-worked values, by torch's E4M3 conversion and by brute force."""

import numpy as np
import pytest
import torch

from oracle import fp8_ref as ref


def test_code_values():
    v = ref.VALUES
    assert v[0x00] == 0.0 and v[0x01] == 2.0 ** -9 and v[0x07] == 7 * 2.0 ** -9
    assert v[0x08] == 2.0 ** -6 and v[0x38] == 1.0 and v[0x3C] == 1.5 and v[0x7E] == 448.0
    assert v[0xB8] == -1.0 and np.isnan(v[0x7F]) and np.isnan(v[0xFF])
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, t, equal_nan=True)


def test_rounding():
    # ties go to the even code: 17 lies between 16 (code 0x58) and 18 (0x59), 19 between 18 and 20
    assert list(ref.VALUES[ref.e4m3_codes([17.0, 19.0, -17.0, 460.0, 2.0 ** -10, 1.5 * 2.0 ** -9])]) \
        == [16.0, 20.0, -16.0, 448.0, 0.0, 2 * 2.0 ** -9]
    x = np.random.default_rng(0).normal(size=20000) * np.exp2(
        np.random.default_rng(1).integers(-12, 8, 20000))
    x = np.clip(x, -448, 448).astype(np.float32)
    t = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_codes(x), t)


def test_quantize_blocks():
    x = np.zeros((3, 200), np.float32)
    x[0, :128] = 448.0
    x[0, 130] = -7.0
    x[1, 5] = np.inf
    x[2, 199] = 2.0 ** -20
    codes, scales = ref.quantize(x)
    assert scales.shape == (3, 2) and scales[0, 0] == 1.0 and scales[0, 1] == np.float32(7 / 448)
    assert (codes[0, :128] == 0x7E).all() and codes[0, 130] == 0xFE
    assert np.isnan(scales[1, 0]) and (codes[1, :128] == 0).all() and not np.isnan(scales[1, 1])
    assert scales[2, 0] == np.float32(2.0 ** -126) and codes[2, 199] == 0x7E
    whole, s = ref.quantize(x[[0, 2]], 128)
    assert s.shape == (1, 2) and s[0, 0] == 1.0 and (whole[1] == 0).sum() == 200
    v = ref.values(codes[[0]], scales[[0]])
    assert v[0, 0] == 448.0 and abs(v[0, 130] + 7.0) < 1e-6


@pytest.mark.parametrize("align", [1, 4])
def test_sort_and_back(align):
    ids = np.array([[2, 0], [0, -1], [5, 2], [0, 2]])
    offsets, row_slot, slot_row = ref.sort_by_expert(ids, 3, align, 16)
    if align == 1:
        assert list(offsets) == [0, 3, 3, 6]
        assert list(row_slot) == [1, 2, 6, 0, 5, 7] + [-1] * 10
        assert slot_row.tolist() == [[3, 0], [1, -1], [-1, 4], [2, 5]]
    else:
        assert list(offsets) == [0, 4, 4, 8] and list(row_slot[:8]) == [1, 2, 6, -1, 0, 5, 7, -1]
    x = np.random.default_rng(2).normal(size=(4, 5))
    w = np.random.default_rng(3).normal(size=(4, 2))
    rows = ref.dispatch(x, row_slot, 2)
    y, _ = ref.combine(rows, slot_row, w)
    kept = (ids >= 0) & (ids < 3)
    assert np.allclose(y, x * (w * kept).sum(1, keepdims=True))


def test_combine_gradient_by_differences():
    rng = np.random.default_rng(4)
    ids = np.array([[1, 0], [-1, 1], [-1, -1]])
    _, row_slot, slot_row = ref.sort_by_expert(ids, 2, 2, 6)
    y, w, dd = rng.normal(size=(6, 3)), rng.normal(size=(3, 2)), rng.normal(size=(3, 3))
    dy, dw = ref.combine_backward(dd, y, slot_row, 6, w)

    def loss(yy, ww):
        return (ref.combine(yy, slot_row, ww)[0] * dd).sum()
    h = 1e-6
    for grad, arr, f in ((dy, y, lambda v: loss(v, w)), (dw, w, lambda v: loss(y, v))):
        for i in np.ndindex(arr.shape):
            d = np.zeros(arr.shape)
            d[i] = h
            assert abs((f(arr + d) - f(arr - d)) / (2 * h) - grad[i]) < 1e-7
