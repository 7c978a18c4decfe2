"""Stacks of matrices of one row whose rows lie in wider buffers: the pitch is then the stride
from one matrix to the next, whatever the stride of the dimension of one says."""

import numpy as np
import pytest
import torch

from oracle import fp8_ref, nvf4_ref as ref
from test_gpu_moe_layer import Case
from test_gpu_nvf4 import check, dg, gpu, operand, rows16, same  # noqa: F401

pytestmark = pytest.mark.gpu


def wider(t, pad):
    """t [count, 1, n] with its rows pad further apart, as a view of a [count, n] one."""
    room = torch.empty(t.shape[0], t.stride(0) + pad, dtype=t.dtype, device="cuda")
    return room[:, :t.shape[2]].copy_(t[:, 0])[:, None]


@pytest.mark.parametrize("pad", [16, 80])
def test_quantize_and_back(dg, pad):  # noqa: F811
    count, K = 5, 100
    x, x64 = rows16(count, K, 1, "bf16")
    codes, scales, rows = dg.nvf4_buffers(count, 1, K)
    out = (wider(codes, pad), scales, rows)
    dg.quantize_nvf4(x[:, None], out=out)
    d = wider(torch.empty(count, 1, K, device="cuda"), 3)
    dg.dequantize_nvf4(*out, d)
    for z in range(count):
        want = ref.quantize(x64[z:z + 1])
        assert same([t[z] for t in out], want)
        assert np.array_equal(d[z].double().cpu().numpy(), ref.values(*want))


@pytest.mark.parametrize("pad", [16, 80])
def test_grouped(dg, pad):  # noqa: F811
    count, K = 3, 200
    a, av = operand(384, K, 2)
    parts = [operand(1, K, 3 + e) for e in range(count)]
    codes, scales, rows = [torch.stack([p[0][i].view(torch.uint8) if i == 1 else p[0][i]
                                        for p in parts]) for i in range(3)]
    room = torch.empty(count, 112 + pad, dtype=torch.uint8, device="cuda")
    room[:, :K // 2] = codes[:, 0]
    d = torch.empty(384, 1, device="cuda")
    dg.gemm_nvf4_grouped(*a, room[:, None, :K // 2], scales.view(torch.float8_e4m3fn), rows,
                         gpu(np.array([0, 128, 256, 384], np.int32)), d)
    for e in range(count):
        at = slice(128 * e, 128 * e + 128)
        check(d[at], *ref.product(av[at], parts[e][1]), "f32")
    dg.check_status()


@pytest.mark.parametrize("fmt", ["fp8", "nvf4"])
@pytest.mark.parametrize("what", ["up", "down"])
def test_layer(dg, fmt, what):  # noqa: F811
    hidden, out = (1, 40) if what == "up" else (40, 1)
    c = Case(fmt, 3, 2, 4, 72, hidden, out, "f16", seed=6)
    w = getattr(c, what)
    room = torch.zeros(4, 144, dtype=torch.uint8, device="cuda")
    width = w[0].shape[2]
    room[:, :width] = w[0].view(torch.uint8)[:, 0]
    setattr(c, what, (room[:, :width][:, None].view(w[0].dtype),) + w[1:])
    c.run(dg)
    c.check()
    dg.check_status()
