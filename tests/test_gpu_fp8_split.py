"""FP8 products of few tiles: divided along K over clusters of CTAs where that
saves more than the cluster costs, whole where it does not."""

import pytest
import torch

from oracle import fp8_ref as ref
from test_gpu_fp8 import TYPES, check, dg, operand  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,block_rows", [
    (64, 8000, 1280, 128), (64, 8000, 2048, 128), (64, 4096, 1280, 128), (64, 4096, 2048, 128),
    (256, 4096, 2560, 128), (64, 8000, 2304, 1), (64, 4096, 1536, 1)])
def test_short_k_is_not_split(dg, M, N, K, block_rows):  # noqa: F811
    """Its sums have the bits of a product of many rows, whose tiles fill the
    SMs and are whole: both add the blocks of K in their order."""
    a, sa, _ = operand(M, K, 91)
    b, sb, _ = operand(N, K, 92, block_rows, scale=0.05)
    few = torch.empty(M, N, device="cuda")
    dg.gemm_fp8(a, sa, b, sb, few)
    times = 2048 // M
    many = torch.empty(times * M, N, device="cuda")
    dg.gemm_fp8(a.view(torch.uint8).repeat(times, 1).view(a.dtype), sa.repeat(times, 1), b, sb, many)
    dg.check_status()
    assert torch.equal(many, few.repeat(times, 1))


@pytest.mark.parametrize("epilogue,beta", [("none", 0.0), ("bias_gelu", 0.0), ("bias", -0.5)])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,N,K", [(300, 2000, 5000),   # halves
                                   (65, 2001, 5123),    # quarters
                                   (140, 1030, 2900)])  # quarters, the last of them empty
def test_split(dg, M, N, K, block_rows, epilogue, beta):  # noqa: F811
    a, sa, av = operand(M, K, 93)
    b, sb, bv = operand(N, K, 94, block_rows, scale=0.05)
    g = torch.Generator().manual_seed(95)
    for dtype in ("f16", "bf16", "f32"):
        t = TYPES[dtype]
        bias = torch.randn(N, generator=g).to(t)
        room = torch.randn(M, (N + 7) // 8 * 8 + 8, generator=g).to(t).cuda()
        before = room.clone()
        dg.gemm_fp8(a, sa, b, sb, room[:, :N], bias=bias.cuda(), beta=beta, epilogue=epilogue)
        dg.check_status()
        check(room[:, :N], *ref.product(
            av, bv, beta=beta, d=before[:, :N].double().cpu().numpy(), use_gelu="gelu" in epilogue,
            bias=bias.double().numpy() if "bias" in epilogue else None), dtype)
        assert torch.equal(room[:, N:], before[:, N:])
