"""FP8 products per expert at the sizes of prompts: 128 x 256 tiles, several to
a CTA, whose pipelines, scale groups and output boxes carry on from one tile and
expert to the next, and more experts than a warp's lanes."""

import numpy as np
import pytest
import torch

from oracle import fp8_ref as ref
from test_gpu_fp8 import TYPES, check, dg, expert_weights, gpu, operand  # noqa: F401

pytestmark = pytest.mark.gpu


def segments(kind):
    rng = np.random.default_rng(7)
    if kind == "prompt":  # some empty, few a multiple of 128
        return [0, 301, 128, 0, 517, 1, 640, 255, 0, 333, 129, 384, 470, 0, 97, 700]
    if kind == "64":
        return [int(v) for v in rng.integers(0, 121, 64)]
    return [0] * 40 + [int(v) for v in rng.integers(0, 90, 93)] + [300, 0]


def tiles(sizes, rows, N, bn, sms):
    """The launch's rounds over the SMs as its rule counts them, and the tiles there are."""
    blocks = rows // 128 + min(len(sizes), rows)
    n = -(-N // bn)
    return -(-blocks * n // sms), sum(-(-s // 128) for s in sizes) * n


@pytest.fixture(scope="module")
def prepared():
    kept = {}

    def get(kind, N, K):
        if (kind, N, K) not in kept:
            kept.clear()
            sizes = segments(kind)
            kept[kind, N, K] = sizes, operand(sum(sizes) + 3, K, 81), \
                expert_weights(len(sizes), N, K, 82)
        return kept[kind, N, K]
    return get


@pytest.mark.parametrize("kind,N,K,dtype,epilogue,beta", [
    ("prompt", 1500, 400, "f16", "bias_gelu", 0.0),
    ("prompt", 1500, 400, "bf16", "none", 0.0),
    ("prompt", 1500, 400, "f32", "gelu", 0.0),
    ("prompt", 1500, 400, "f32", "bias", -0.5),
    ("prompt", 1504, 400, "f16", "none", 0.0),
    ("prompt", 1504, 400, "bf16", "bias_gelu", 0.0),
    ("prompt", 1504, 400, "f32", "none", 0.0),
    ("prompt", 1504, 400, "f16", "bias_gelu", 0.5),
    ("prompt", 1504, 400, "f32", "gelu", 0.5),
    ("64", 520, 1100, "f16", "bias_gelu", 0.0),
    ("64", 520, 1100, "bf16", "none", 0.25),
    ("64", 517, 1100, "f32", "bias", 0.0),
    ("135", 100, 700, "f32", "bias", 0.0),
    ("135", 100, 700, "bf16", "gelu", 0.5),
])
def test_grouped_tiles(dg, prepared, kind, N, K, dtype, epilogue, beta):  # noqa: F811
    sizes, (a, sa, av), (b, sb, bv) = prepared(kind, N, K)
    used, rows = sum(sizes), sum(sizes) + 3
    sms = dg.query_hw().sm_count
    assert rows > 16 * len(sizes)  # more rows than the few-rows kernel takes
    if kind != "135":
        wide, there = tiles(sizes, rows, N, 256, sms)
        assert wide < tiles(sizes, rows, N, 128, sms)[0] and there > sms
    t = TYPES[dtype]
    g = torch.Generator().manual_seed(83)
    bias = torch.randn(len(sizes), N, generator=g).to(t)
    room = torch.randn(rows, (N + 7) // 8 * 8 + 8, generator=g).to(t).cuda()
    before = room.clone()
    dg.gemm_fp8_grouped(a, sa, b, sb, gpu(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)),
                        room[:, :N], bias=bias.cuda(), alpha=0.75, beta=beta, epilogue=epilogue)
    dg.check_status()
    assert torch.equal(room[used:], before[used:]) and torch.equal(room[:, N:], before[:, N:])
    end = 0
    for e, size in enumerate(sizes):
        at, end = slice(end, end + size), end + size
        if size:
            check(room[at, :N], *ref.product(
                av[at], bv[e], alpha=0.75, beta=beta, d=before[at, :N].double().cpu().numpy(),
                use_gelu="gelu" in epilogue,
                bias=bias[e].double().numpy() if "bias" in epilogue else None), dtype)
