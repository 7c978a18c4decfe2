"""The NVF4 operators and the expert layer on rows and matrices that lie so far apart
that their offsets do not fit 32 bits."""

import numpy as np
import pytest
import torch

from oracle import fp8_ref, nvf4_ref as ref
from test_gpu_moe_layer import Case
from test_gpu_nvf4 import check, dg, gpu, operand, rows16, same  # noqa: F401

pytestmark = pytest.mark.gpu

FAR = 2 ** 31 + 1024  # elements, between neighbours


def spread(t, stride):
    """t with its first dimension `stride` elements apart, in a buffer of its own."""
    room = torch.empty(stride * (t.shape[0] - 1) + t[0].numel(), dtype=t.dtype, device="cuda")
    far = room.as_strided(t.shape, (stride,) + t[0].contiguous().stride())
    return far.copy_(t)


@pytest.mark.parametrize("stack", [False, True])
def test_quantize_and_back(dg, stack):  # noqa: F811
    K = 72
    x, x64 = rows16(3, K, 50, "bf16")
    want = ref.quantize(x64)
    far = spread(x, FAR)
    codes = torch.empty(2 * FAR + 48, dtype=torch.uint8, device="cuda").as_strided((3, 36), (FAR, 1))
    scales = torch.empty((1, 2, 32, 16), dtype=torch.uint8, device="cuda")
    rows = torch.empty(3, device="cuda")
    if stack:
        far, codes = far[:, None], codes[:, None]
        scales, rows = scales.expand(3, 1, 2, 32, 16).contiguous(), rows[:, None]
    out = (codes, scales.view(torch.float8_e4m3fn), rows)
    dg.quantize_nvf4(far, out=out)
    parts = [tuple(v[i] for v in out) for i in range(3)] if stack else [out]
    for i, part in enumerate(parts):
        assert same(part, tuple(v[i:i + 1] for v in want) if stack else want)
    d = torch.empty(2 * FAR + K, dtype=torch.float16, device="cuda").as_strided(
        far.shape, (FAR,) + ((K,) if stack else ()) + (1,))
    dg.dequantize_nvf4(*out, d)
    exact = torch.from_numpy(ref.values(*want)).half().reshape(d.shape)
    assert torch.equal(d.cpu(), exact)


@pytest.mark.parametrize("M", [3, 300])
def test_gemm(dg, M):  # noqa: F811
    K, N = 200, 136
    a, av = operand(M, K, 51)
    b, bv = operand(N, K, 52)
    t, err = ref.product(av, bv)
    apart = FAR if M == 3 else 2 ** 23 + 64  # (300 rows of 2^23 elements)
    fa = spread(a[0], apart)
    d = torch.empty(apart * (M - 1) + N, dtype=torch.float16, device="cuda").as_strided(
        (M, N), (apart, 1))
    check(dg.gemm_nvf4(fa, *a[1:], *b, d), t, err, "f16")


def test_grouped(dg):  # noqa: F811
    K, N = 128, 72
    a, av = operand(256, K, 53)
    parts = [operand(N, K, 54 + e) for e in range(2)]
    codes = spread(torch.stack([p[0][0] for p in parts]), 2 * FAR)
    scales = torch.stack([p[0][1].view(torch.uint8) for p in parts]).view(torch.float8_e4m3fn)
    rows = torch.stack([p[0][2] for p in parts])
    d = torch.empty(256, N, device="cuda")
    dg.gemm_nvf4_grouped(*a, codes, scales, rows, gpu(np.array([0, 128, 256], np.int32)), d)
    for e in range(2):
        t, err = ref.product(av[128 * e:128 * e + 128], parts[e][1])
        check(d[128 * e:128 * e + 128], t, err, "f32")
    dg.check_status()


@pytest.mark.parametrize("fmt", ["fp8", "nvf4"])
def test_layer(dg, fmt):  # noqa: F811
    # weights, biases, tokens and results
    c = Case(fmt, 3, 2, 2, 128, 128, 128, bias=True, gated=True, seed=55)
    c.up = (spread(c.up[0].contiguous().view(torch.uint8), 2 * FAR).view(c.up[0].dtype),) + c.up[1:]
    c.down = (spread(c.down[0].contiguous().view(torch.uint8), 2 * FAR).view(c.down[0].dtype),) + \
        c.down[1:]
    c.bias = [spread(v, FAR) for v in c.bias]
    c.x = spread(c.x, FAR)
    c.d = torch.empty(2 * FAR + 128, dtype=c.d.dtype, device="cuda").as_strided((3, 128), (FAR, 1))
    c.run(dg)
    dg.check_status()
    y, bound = c.wanted()
    assert (np.abs(c.d.double().cpu().numpy() - y) <= bound).all()
