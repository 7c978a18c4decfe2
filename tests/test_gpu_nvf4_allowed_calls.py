"""Calls of the NVF4 operators and the expert layer that include/dg.h allows at their edges:
nothing to do, factors that are zero, infinite or NaN, one bias for all experts, scales in wider
rows, results over the tokens, several threads at once."""

import threading

import numpy as np
import pytest
import torch

from oracle import fp8_ref, nvf4_ref as ref
from test_gpu_moe_layer import Case
from test_gpu_nvf4 import check, dg, gpu, operand  # noqa: F401

pytestmark = pytest.mark.gpu


def test_nothing_to_do(dg):  # noqa: F811
    for shape in ((0, 64), (5, 0), (0, 5, 64), (3, 0, 64), (3, 5, 0)):
        x = torch.empty(shape, dtype=torch.float16, device="cuda")
        q = dg.quantize_nvf4(x)
        assert q[0].shape[:-1] == shape[:-1]
        assert dg.dequantize_nvf4(*q, torch.empty_like(x)).shape == shape
    a, b = operand(4, 64, 1)[0], operand(8, 64, 2)[0]
    none = dg.nvf4_buffers(0, 64)
    dg.gemm_nvf4(*none, *b, torch.empty(0, 8, device="cuda"))
    dg.gemm_nvf4(*a, *none, torch.empty(4, 0, device="cuda"))
    offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    dg.gemm_nvf4_grouped(*none, *dg.nvf4_buffers(2, 8, 64), offsets, torch.empty(0, 8, device="cuda"))
    # no token at all, and rows without one
    slots = torch.full((130,), -1, dtype=torch.int32, device="cuda")
    q = dg.moe_dispatch_nvf4(torch.empty(0, 64, dtype=torch.float16, device="cuda"), slots, 2,
                             *dg.nvf4_buffers(130, 64))
    assert (dg.dequantize_nvf4(*q, torch.ones(130, 64, device="cuda")) == 0).all()
    dg.moe_dispatch_nvf4(torch.ones(3, 64, dtype=torch.float16, device="cuda"), slots[:0], 2,
                         *dg.nvf4_buffers(0, 64))
    c = Case("nvf4", 2, 2, 3, 64, 64, 64, "f16")
    dg.moe_layer(c.x[:0], c.ids[:0], c.w[:0], c.up, c.down, c.d[:0])
    dg.check_status()


@pytest.mark.parametrize("M,N", [(20, 100), (300, 2900)])
def test_odd_factors(dg, M, N):  # noqa: F811
    K = 192
    (ac, asc, ar), av = operand(M, K, 3)
    (bc, bsc, br), bv = operand(N, K, 4)
    ar, br = ar.clone(), br.clone()
    ar[3], ar[5], ar[7], br[2], br[9] = 0.0, float("nan"), float("inf"), 0.0, float("nan")
    av[3] = 0.0
    bv[2] = 0.0
    t, err = ref.product(av, bv)
    d = dg.gemm_nvf4(ac, asc, ar, bc, bsc, br, torch.empty(M, N, device="cuda"))
    assert torch.isnan(d[5]).all() and torch.isnan(d[:, 9]).all()
    assert torch.isnan(d[7, 2])  # infinity times zero
    finite = np.ones((M, N), bool)
    finite[[5, 7]] = False
    finite[:, 9] = False
    g = d.double().cpu().numpy()
    assert (np.abs(g - t) <= fp8_ref.rounded_bound(t, err, "f32"))[finite].all()
    assert (g[3][finite[3]] == 0).all() and (g[:, 2][finite[:, 2]] == 0).all()
    # alpha 0: beta * D and the bias alone
    c = torch.randn(M, N, device="cuda")
    bias = torch.randn(N, device="cuda")
    (a, _), (b, _) = operand(M, K, 5), operand(N, K, 6)
    want = (0.5 * c.double() + bias.double()).cpu().numpy()
    d = dg.gemm_nvf4(*a, *b, c, bias=bias, alpha=0.0, beta=0.5, epilogue="bias")
    assert (np.abs(d.double().cpu().numpy() - want) <= np.abs(want) * 2.0 ** -24 + 1e-45).all()


@pytest.mark.parametrize("fmt", ["fp8", "nvf4"])
def test_one_bias_for_all_experts(dg, fmt):  # noqa: F811
    c = Case(fmt, 3, 2, 4, 96, 128, 72, "bf16", bias=True, seed=7)
    c.bias = [b[:1].clone().expand(4, -1) for b in c.bias]
    c.bias64 = tuple(np.repeat(b[:1], 4, 0) for b in c.bias64)
    c.run(dg)
    c.check()


def test_layer_scales_in_wider_rows(dg):  # noqa: F811
    c = Case("fp8", 4, 2, 3, 300, 200, 136, "f16", seed=8)
    for name in ("up", "down"):
        codes, s = getattr(c, name)
        room = torch.full((3, s.shape[1] + 1, s.shape[2] + 3), float("nan"), device="cuda")
        room[:, :s.shape[1], :s.shape[2]] = s
        setattr(c, name, (codes, room[:, :s.shape[1], :s.shape[2]]))
    c.run(dg)
    c.check()


@pytest.mark.parametrize("fmt", ["fp8", "nvf4"])
@pytest.mark.parametrize("tokens", [1, 6])
def test_results_over_the_tokens(dg, fmt, tokens):  # noqa: F811
    c = Case(fmt, tokens, 2, 4, 256, 128, 256, "bf16", seed=9)
    c.d = c.x
    c.room = c.x
    y, bound = c.wanted()
    c.run(dg)
    assert (np.abs(c.x.double().cpu().numpy() - y) <= bound).all()


def test_threads(dg):  # noqa: F811
    """Layers and products of several host threads, each on a stream of its own."""
    cases = [Case("nvf4" if i % 2 else "fp8", 4, 2, 8, 512, 256, 512, "bf16", True, seed=20 + i)
             for i in range(6)]
    a, av = operand(300, 512, 30)
    b, bv = operand(200, 512, 31)
    out = [torch.empty(300, 200, device="cuda") for _ in cases]
    torch.cuda.synchronize()
    failed = []

    def work(c, d):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(30):
                    c.run(dg)
                    dg.gemm_nvf4(*a, *b, d)
            s.synchronize()
        except Exception as e:  # (a thread's exception ends nothing else)
            failed.append(e)
    threads = [threading.Thread(target=work, args=v) for v in zip(cases, out)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for c in cases:
        c.check()
    t, err = ref.product(av, bv)
    for d in out:
        check(d, t, err, "f32")
    dg.check_status()
