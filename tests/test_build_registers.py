"""The build fails where ptxas gives a kernel with divided registers another
count than its warpgroups' shares add up to (else only its launch would)."""

import pytest

from precision_matmul_dg_gb300 import build

SOURCE = "constexpr int kLaunchRegs = 168, kSumRegs = 216, kOtherRegs = 72;"
LINE = "ptxas info    : Used %d registers, used 1 barriers\n"


def test_registers():
    build.check_registers("x.cu", SOURCE, LINE % 168 + "other\n" + LINE % 168)
    for out in (LINE % 168 + LINE % 160, LINE % 160, ""):
        with pytest.raises(RuntimeError, match="168"):
            build.check_registers("x.cu", SOURCE, out)


def test_sources_name_their_count():
    import os
    for src in build.FIXED_REGS:
        text = open(os.path.join(build.CSRC, src)).read()
        with pytest.raises(RuntimeError):
            build.check_registers(src, text, LINE % 1)
