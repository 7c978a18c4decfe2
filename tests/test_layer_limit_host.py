"""The expert layer's limit of tokens, experts and slots, as include/dg.h states it: sizes at
the limit are accepted (and refused only for their missing scratch), one step more is not."""

import ctypes
import os
import re

import pytest

from test_nvf4_host import dg  # noqa: F401

P = 0x10000
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dg.h")


def taken(tokens, top_k, count, width):
    """Bytes by dg.h's formula."""
    return 68 * tokens + 2 * tokens * (-(-width // 256) * 256) + 12 * count + 24 * tokens * top_k


# what dg.h leaves of the 150 KiB
LESS = int(re.search(r"24 for each slot are at most 150 KiB, less (\d+)\)",
                     re.sub(r"[\s*]+", " ", open(HEADER).read())).group(1))


def error(dg, tokens, top_k, count, width):  # noqa: F811
    ld = -(-width // 16) * 16
    lds = -(-width // 128)
    up = dg.MoeWeights(P, ld, 16 * ld, P, lds, lds, None, None, 0)
    down = dg.MoeWeights(P, 16, 16 * 16, P, 1, 1, None, None, 0)
    status = dg.lib().dg_moe_layer(tokens, top_k, count, width, 16, 16, dg.F16, P, ld, P, P, 0,
                                   ctypes.byref(up), ctypes.byref(down), 0, P, 16, None, 0, None)
    assert status != 0
    return dg.last_error()


@pytest.mark.parametrize("top_k,count,width", [(8, 256, 7168), (8, 256, 4096), (1, 4, 2048),
                                               (2, 1024, 256), (2, 1023, 200), (3, 64, 1000),
                                               (1, 1, 8500), (4, 17, 5120)])
def test_tokens(dg, top_k, count, width):  # noqa: F811
    fits = max(t for t in range(1, 512 // top_k + 1)
               if taken(t, top_k, count, width) <= 150 * 1024 - LESS)
    assert "scratch" in error(dg, fits, top_k, count, width)
    assert "shared memory" in error(dg, fits + 1, top_k, count, width)


def test_experts(dg):  # noqa: F811
    # sizes where the count of experts alone decides, and one exactly at the limit
    found = exact = 0
    for width in range(256, 4096, 256):
        for top_k in (1, 2, 3, 5):
            for tokens in range(1, 512 // top_k + 1):
                room = 150 * 1024 - LESS - taken(tokens, top_k, 0, width)
                count = room // 12
                if 1 <= count < 1024:
                    found += 1
                    exact += room % 12 == 0
                    if found % 7 == 0 or room % 12 == 0:
                        assert "scratch" in error(dg, tokens, top_k, count, width)
                        assert "shared memory" in error(dg, tokens, top_k, count + 1, width)
    assert found > 10 and exact > 0
