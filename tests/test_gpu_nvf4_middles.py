"""Quantization of values in the middle between two codes, and one step beside it, for every
block scale, at row scales over the whole range of the type."""

import numpy as np
import pytest
import torch

from oracle import fp8_ref, nvf4_ref as ref
from test_gpu_nvf4 import TYPES, dg, same  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,exponent", [("f16", -5), ("f16", 4), ("bf16", -100), ("bf16", -99),
                                            ("bf16", -50), ("bf16", -1), ("bf16", 31),
                                            ("bf16", 100), ("bf16", 116)])
def test_middles_of_all_scales(dg, dtype, exponent):  # noqa: F811
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    rows = np.zeros((126, 80))
    for s in range(1, 127):
        v = mids * fp8_ref.VALUES[s]
        rows[s - 1, :8], rows[s - 1, 8:16] = v, -v
        # (the largest value of these blocks is as above: their scale is the same)
        rows[s - 1, 16:23] = v[:7] * (1 + 2.0 ** -7)
        rows[s - 1, 24:31] = -v[:7] * (1 + 2.0 ** -7)
        rows[s - 1, 32:39] = v[:7] * (1 - 2.0 ** -8)
        rows[s - 1, 40:47] = -v[:7] * (1 - 2.0 ** -8)
        rows[s - 1, [23, 31, 39, 47]] = v[7]
    rows[:, 64] = 2688.0
    x = torch.from_numpy(rows * 2.0 ** exponent).to(TYPES[dtype])
    assert torch.isfinite(x).all()
    want = ref.quantize(x.double().numpy())
    assert (want[2] == 2.0 ** exponent).all()
    if dtype == "bf16":  # (exact there; the smallest of FP16 are rounded)
        assert np.array_equal(want[1][:, :3], np.repeat(np.arange(1, 127)[:, None], 3, 1))
    assert same(dg.quantize_nvf4(x.cuda()), want)
