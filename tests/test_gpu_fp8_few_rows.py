"""Where FP8 products pass from the few-rows kernel to the tensor-core kernel:
right on both sides, and on the tensor-core side where that one is faster."""

import numpy as np
import pytest
import torch

from oracle import fp8_ref as ref
from test_gpu_fp8 import check, dg, expert_weights, gpu, operand  # noqa: F401

pytestmark = pytest.mark.gpu


def padded(codes, K):
    """Contiguous bytes as codes in rows that start on 16-byte boundaries."""
    wide = torch.full((codes.shape[0], (K + 15) // 16 * 16), 0x7F, dtype=torch.uint8, device="cuda")
    wide[:, :K] = codes
    return wide.view(torch.float8_e4m3fn)[:, :K]


@pytest.mark.parametrize("M,N,K", [(32, 8960, 1536), (17, 5000, 512), (16, 9800, 1000)])
def test_rows_of_a_dense_product(dg, M, N, K):  # noqa: F811
    # the bits of the same rows among 2000, which the tensor-core kernel multiplies
    a, sa, _ = operand(M, K, 101)
    b, sb, _ = operand(N, K, 102, 128, scale=0.05)
    few = torch.empty(M, N, device="cuda")
    dg.gemm_fp8(a, sa, b, sb, few)
    times = 2000 // M
    many = torch.empty(times * M, N, device="cuda")
    dg.gemm_fp8(padded(a.view(torch.uint8).repeat(times, 1), K), sa.repeat(times, 1), b, sb, many)
    dg.check_status()
    assert torch.equal(many, few.repeat(times, 1))


def test_rows_of_experts(dg):  # noqa: F811
    # eight to an expert: the bits of the same rows among 160
    count, N, K = 64, 520, 700
    a, sa, _ = operand(8 * count, K, 103)
    b, sb, _ = expert_weights(count, N, K, 104)
    few = torch.empty(8 * count, N, device="cuda")
    dg.gemm_fp8_grouped(a, sa, b, sb, gpu(np.arange(count + 1, dtype=np.int32) * 8), few)
    many = torch.empty(160 * count, N, device="cuda")

    def spread(t):
        return t.reshape(count, 8, -1).repeat(1, 20, 1).reshape(160 * count, -1)
    dg.gemm_fp8_grouped(padded(spread(a.view(torch.uint8)), K), spread(sa), b, sb,
                        gpu(np.arange(count + 1, dtype=np.int32) * 160), many)
    dg.check_status()
    assert torch.equal(many, spread(few))


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,N,K", [(8, 9900, 260), (9, 9900, 260), (16, 9700, 260), (16, 9900, 130),
                                   (17, 2400, 1030), (32, 4800, 400), (32, 4900, 400), (31, 9900, 130),
                                   (24, 4096, 4096), (25, 4096, 4224)])
def test_dense_on_both_sides(dg, M, N, K, block_rows):  # noqa: F811
    a, sa, av = operand(M, K, 105)
    b, sb, bv = operand(N, K, 106, block_rows, scale=0.05)
    d = torch.full((M, N), float("nan"), device="cuda")
    dg.gemm_fp8(a, sa, b, sb, d)
    dg.check_status()
    check(d, *ref.product(av, bv), "f32")


@pytest.mark.parametrize("N,K", [(72, 700), (1100, 260), (5000, 130)])
@pytest.mark.parametrize("sizes", [[25], [12] * 6, [1, 30, 0, 9, 20, 12], [3, 0, 9, 1, 7, 0, 30, 2],
                                   [5] * 20, [0, 33]])
def test_experts_on_both_sides(dg, sizes, N, K):  # noqa: F811
    rows = sum(sizes)
    a, sa, av = operand(rows, K, 107)
    b, sb, bv = expert_weights(len(sizes), N, K, 108)
    d = torch.full((rows, N), float("nan"), device="cuda")
    ends = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    dg.gemm_fp8_grouped(a, sa, b, sb, gpu(ends), d)
    dg.check_status()
    for e in range(len(sizes)):
        at = slice(ends[e], ends[e + 1])
        if sizes[e]:
            check(d[at], *ref.product(av[at], bv[e]), "f32")


def test_offsets_are_clamped_with_few_rows(dg):  # noqa: F811
    b, sb, bv = expert_weights(3, 64, 128, 42)
    a, sa, av = operand(30, 128, 41)
    d = torch.full((30, 64), 7.0, device="cuda")
    dg.gemm_fp8_grouped(a, sa, b, sb, gpu(np.array([-5, 10, 4, 1000], np.int32)), d)
    dg.check_status()
    check(d[:4], *[x[:4] for x in ref.product(av[:4], bv[0])], "f32")
    check(d[10:], *ref.product(av[10:], bv[2]), "f32")
