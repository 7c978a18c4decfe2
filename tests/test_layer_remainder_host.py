"""The layer of layer_remainder.py, within the bound of oracle.nvf4_ref.layer as h is held and
outside it with the second value of h lost or another's."""

import numpy as np
import pytest

from layer_remainder import Layer
from oracle import fp8_ref, nvf4_ref as ref


@pytest.mark.parametrize("gated", [False, True])
def test_what_is_found(gated):
    c = Layer(gated=gated)
    y, err = ref.layer(c.x, c.ids, None, c.up, c.down, gated)
    bound = fp8_ref.rounded_bound(y, err, "f16")
    exact = c.results(np.array([c.h(t) for t in range(len(c.x))]))
    assert np.abs(y - exact).max() < 1e-9
    # two FP16 values hold all of h
    assert np.array_equal(c.results(c.held()), exact)
    groups = c.hidden // 32
    for mistake in ("bits", "slot", "power"):
        d = c.results(c.held(mistake)).astype(np.float16)
        bad = np.abs(d - y) > bound
        # in every token, and every group (whose neighbour has another power: all)
        assert bad.reshape(len(c.x), groups, 32).any(2).all(), mistake
        # and at every place among the 32
        assert bad.reshape(len(c.x), groups, 32).any((0, 1)).all(), mistake
