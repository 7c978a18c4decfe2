"""The expert layer's hidden values in 22 bits: results that are differences of hidden values
whose first 11 bits agree (layer_remainder.py)."""

import numpy as np
import pytest
import torch

from layer_remainder import Layer
from oracle import fp8_ref, nvf4_ref as ref
from test_gpu_moe_layer import TYPES, dg, gpu  # noqa: F401

pytestmark = pytest.mark.gpu


def stack(fmt, values):
    """Matrices of codes' values with all scales 1, on the GPU."""
    count, n, k = values.shape
    if fmt == "fp8":
        codes = torch.from_numpy(values).float().to(torch.float8_e4m3fn)
        room = torch.zeros(count, n, -(-k // 16) * 16, dtype=torch.uint8, device="cuda")
        room[..., :k] = codes.view(torch.uint8).cuda()
        return (room.view(torch.float8_e4m3fn)[..., :k],
                torch.ones(count, -(-n // 128), -(-k // 128), device="cuda"))
    one = fp8_ref.e4m3_codes(np.ones((n, -(-k // 16))))
    room = torch.zeros(count, n, -(-k // 32) * 16, dtype=torch.uint8, device="cuda")
    room[..., :k // 2] = gpu(np.stack([ref.pack(ref.e2m1_codes(v)) for v in values]))
    return (room[..., :k // 2],
            gpu(np.stack([ref.tiles(one)] * count)).view(torch.float8_e4m3fn),
            torch.ones(count, n, device="cuda"))


@pytest.mark.parametrize("fmt", ["fp8", "nvf4"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tokens,hidden", [(1, 128), (7, 1152), (14, 2432)])
def test_differences_of_hidden_values(dg, fmt, gated, dtype, tokens, hidden):  # noqa: F811
    c = Layer(tokens=tokens, hidden=hidden, gated=gated, seed=tokens)
    x = torch.from_numpy(c.x).to(TYPES[dtype])
    assert np.array_equal(x.double().numpy(), c.x)
    d = torch.empty(tokens, hidden, dtype=x.dtype, device="cuda")
    dg.moe_layer(x.cuda(), gpu(c.ids), None, stack(fmt, c.up), stack(fmt, c.down), d,
                 activation="swiglu" if gated else "gelu")
    dg.check_status()
    y, err = ref.layer(c.x, c.ids, None, c.up, c.down, gated)
    bad = ~(np.abs(d.double().cpu().numpy() - y) <= fp8_ref.rounded_bound(y, err, dtype))
    assert not bad.any(), "%d of %d outside the bound, first at %s" % (
        bad.sum(), bad.size, np.argwhere(bad)[0])
