"""Experts' offsets that go back and forth: segments that overlap so far that their tiles are
more than a 32-bit walk takes.  The count stops there, the status word says so, and nothing is
written outside D."""

import pytest
import torch

from test_gpu_nvf4 import dg  # noqa: F401

pytestmark = pytest.mark.gpu


def test_more_tiles_than_a_walk_takes(dg):  # noqa: F811
    # 512 times all of 4096 rows, in chunks of 8, and 8192 tiles of 64 columns: 2^31 tiles
    count, rows, N, K = 1024, 4096, 1 << 19, 16
    one = torch.full((rows, K), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    w = torch.full((count, N, K), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    offsets = torch.zeros(count + 1, dtype=torch.int32, device="cuda")
    offsets[1::2] = rows
    room = torch.zeros((rows + 2) * N, dtype=torch.float16, device="cuda")
    d = room[N:-N].view(rows, N)
    dg.gemm_fp8_grouped(one, torch.ones(rows, 1, device="cuda"), w,
                        torch.ones(count, N // 128, 1, device="cuda"), offsets, d)
    with pytest.raises(dg.DgError, match="status word 1"):
        dg.check_status()
    assert (d == K).all()
    assert (room[:N] == 0).all() and (room[-N:] == 0).all()


@pytest.mark.parametrize("rows", [24, 4096])
def test_segments_that_overlap(dg, rows):  # noqa: F811
    # every second expert has all rows: each is a legal answer, and the status word is clean
    count, N, K = 66, 160, 128
    w = torch.zeros(count, N, K, dtype=torch.uint8, device="cuda")
    w[0::2, :, 0] = 0x38
    x = torch.full((rows, K), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    offsets = torch.zeros(count + 1, dtype=torch.int32, device="cuda")
    offsets[1::2] = rows
    d = torch.zeros(rows, N, device="cuda")
    dg.gemm_fp8_grouped(x, torch.ones(rows, 1, device="cuda"), w.view(torch.float8_e4m3fn),
                        torch.ones(count, 2, 1, device="cuda"), offsets, d)
    dg.check_status()
    assert (d == 1).all()
    a = dg.quantize_nvf4(torch.ones(rows, K, dtype=torch.float16, device="cuda"))
    b = dg.quantize_nvf4(torch.ones(count, N, K, dtype=torch.float16, device="cuda"))
    d.zero_()
    dg.gemm_nvf4_grouped(*a, *b, offsets, d)
    dg.check_status()
    assert (d > K * 0.9).all() and (d < K * 1.1).all()
