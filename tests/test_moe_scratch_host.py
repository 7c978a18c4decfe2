"""The scratch of dg_moe_dispatch_fp8_ex: its size and its refusals (no GPU)."""

import pytest


@pytest.fixture(scope="module")
def dg():
    import __graft_entry__
    __graft_entry__.build()
    import precision_matmul_dg_gb300 as m
    return m


P = 0x10000  # an aligned address that no check looks behind


def test_size(dg):
    f = dg.lib().dg_moe_dispatch_fp8_scratch
    assert f(640, 8, 2057, 5120) == 640 * (2064 + 4 * 17)
    assert f(640, 8, 2057, 1279) == 0              # fewer than two rows to a token
    assert f(640, 8, 1638, 5120) == 0              # fewer than 2^23 values
    assert f(0, 8, 4096, 1 << 20) == 0
    assert f(1 << 20, 8, 1 << 20, 1 << 23) == (1 << 20) * ((1 << 20) + (1 << 15))  # past 32 bits
    assert f(-1, 8, 64, 8) == -1 and f(1, 0, 64, 8) == -1 and f(1, 1, -1, 8) == -1
    # the binding does not ask below its own limit
    assert dg._SCRATCH_FROM <= 1 << 23
    assert f(640, 8, 1 << 10, (dg._SCRATCH_FROM >> 10) - 1) == 0


def test_refusals(dg):
    def call(scratch, nbytes):
        return dg.lib().dg_moe_dispatch_fp8_ex(640, 8, 2057, 0, P, 2064, 5120, P, P, 2064, P, 17,
                                               scratch, nbytes, None)
    need = 640 * (2064 + 4 * 17)
    for scratch, nbytes, word in ((P, need - 1, "bytes of scratch"), (P, -1, "bytes of scratch"),
                                  (P + 8, need, "16-byte")):
        assert dg.STATUS[call(scratch, nbytes)] == "DG_ERR_INVALID_ARG"
        assert word in dg.last_error()
