"""The expert layer at its limit of shared memory: the largest sizes that include/dg.h admits
run and are right."""

import pytest

from test_gpu_moe_layer import Case, dg  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["fp8", "nvf4"])
@pytest.mark.parametrize("tokens,top_k,count,width,hidden,gated", [
    (225, 2, 1024, 256, 16, False),  # 8 bytes are left
    (236, 1, 921, 256, 24, False),   # none: an expert more is refused
    (36, 1, 4, 2048, 128, True),
    (17, 8, 16, 4096, 128, True),
])
def test_limit(dg, fmt, tokens, top_k, count, width, hidden, gated):  # noqa: F811
    c = Case(fmt, tokens, top_k, count, width, hidden, 24, "bf16", gated, seed=tokens)
    c.run(dg)
    dg.check_status()
    c.check()
