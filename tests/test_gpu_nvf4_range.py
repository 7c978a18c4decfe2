"""NVF4 products and the expert layer where factors of a result lie beyond FP32's range and
their product does not."""

import numpy as np
import pytest
import torch

from oracle import fp8_ref, nvf4_ref as ref
from test_gpu_moe_layer import Case
from test_gpu_nvf4 import TYPES, check, dg, gpu, operand  # noqa: F401

pytestmark = pytest.mark.gpu

LARGEST = {"f32": float(np.finfo(np.float32).max), "bf16": 3.3895313892515355e38}


def scaled(a, values, exponents):
    """An operand with its row scales and values times 2^exponents."""
    f = np.exp2(np.asarray(exponents, np.float64))
    r = (a[2].double().cpu().numpy() * f).astype(np.float32)
    assert np.array_equal(r, a[2].double().cpu().numpy() * f)
    return (a[0], a[1], gpu(r)), values * f[:, None]


def check_finite(got, t, err, dtype):
    """Within the bound where the result is certainly finite, infinite where it is certainly
    beyond; how many are finite and above 2^-60 (others may round to zero)."""
    g = got.double().cpu().numpy()
    top = LARGEST[dtype]
    fine = np.abs(t) + err < top * (1 - 2.0 ** -8)
    bound = fp8_ref.rounded_bound(t, err, dtype)
    bad = fine & ~(np.abs(g - t) <= bound)
    assert not bad.any(), "%d of %d outside the bound, first at %s: %r for %r" % (
        bad.sum(), fine.sum(), np.argwhere(bad)[0], g[bad][0], t[bad][0])
    beyond = np.abs(t) - err > 2.0 ** 128
    assert np.array_equal(g[beyond], np.sign(t[beyond]) * np.inf)
    return (fine & (np.abs(t) > 2.0 ** -60)).sum()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(33, 70), (300, 2900)])
def test_row_scales_that_cancel(dg, M, N, dtype):  # noqa: F811
    K = 320
    rng = np.random.default_rng(M)
    # (operand()'s row scales are within 2^-13 and 2^4)
    a, av = scaled(*operand(M, K, 1), rng.integers(-112, 121, M))
    b, bv = scaled(*operand(N, K, 2), rng.integers(-112, 121, N))
    t, err = ref.product(av, bv)
    d = dg.gemm_nvf4(*a, *b, torch.empty(M, N, dtype=TYPES[dtype], device="cuda"))
    assert check_finite(d, t, err, dtype) > 0.4 * M * N
    # and with all that is added to them
    beta = torch.from_numpy(rng.normal(size=(M, N))).to(TYPES[dtype])
    bias = torch.from_numpy(rng.normal(size=N)).to(TYPES[dtype])
    t, err = ref.product(av, bv, -0.5, 0.25, beta.double().numpy(), bias.double().numpy())
    d = dg.gemm_nvf4(*a, *b, beta.cuda(), bias=bias.cuda(), alpha=-0.5, beta=0.25, epilogue="bias")
    check_finite(d, t, err, dtype)


@pytest.mark.parametrize("pairs", [False, True])
def test_experts_row_scales_that_cancel(dg, pairs):  # noqa: F811
    count, N, K = 2, 200, 128
    rows = 512 * count if pairs else 256
    rng = np.random.default_rng(3)
    a, av = scaled(*operand(rows, K, 4), rng.integers(-112, 121, rows))
    parts = [scaled(*operand(N, K, 5 + e), rng.integers(-112, 121, N)) for e in range(count)]
    b = [torch.stack([p[0][i].view(torch.uint8) if i == 1 else p[0][i] for p in parts])
         for i in range(3)]
    ends = np.array([0, rows // 2, rows], np.int32)
    d = torch.empty(rows, N, device="cuda")
    dg.gemm_nvf4_grouped(*a, b[0], b[1].view(torch.float8_e4m3fn), b[2], gpu(ends), d)
    for e in range(count):
        at = slice(ends[e], ends[e + 1])
        t, err = ref.product(av[at], parts[e][1])
        assert check_finite(d[at], t, err, "f32") > 0.3 * t.size
    dg.check_status()


@pytest.mark.parametrize("gated", [False, True])
def test_layer_of_tiny_tokens(dg, gated):  # noqa: F811
    """Tokens near 2^-117 and row scales of W1 far below one: a row's scale times the power of
    two that a token is held with is below FP32's normal range, the hidden values are not (all
    products have one sign, so they are large against their factors)."""
    c = Case("nvf4", 3, 2, 4, 512, 128, 64, "bf16", gated=False, seed=8)
    c.gated = gated
    if gated:
        c = Case("nvf4", 3, 2, 4, 512, 128, 64, "bf16", gated=True, seed=8)
    tiny = 2.0 ** -117
    x = np.abs(c.x64) + 1.0
    c.x.copy_(torch.from_numpy(x * tiny).to(c.x.dtype))
    c.x64 = c.x.double().cpu().numpy()
    c.up[0].bitwise_and_(0x77)  # W1's codes without their signs
    c.up64 = np.abs(c.up64)
    low = 2.0 ** -9
    rows = slice(128, None) if gated else slice(None)
    if gated:
        # the gates are 2^10 and more times their own scales: SiLU is their argument
        c.up[2][:, :128].mul_(2.0 ** 126)
        c.up64[:, :128] *= 2.0 ** 126
    c.up[2][:, rows].mul_(low)
    c.up64[:, rows] *= low
    lift = 2.0 ** 100
    c.down[2].mul_(lift)
    c.down64 = c.down64 * lift
    c.run(dg)
    c.check()
