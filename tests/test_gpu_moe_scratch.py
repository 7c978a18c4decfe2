"""dg_moe_dispatch_fp8 where the tokens are quantized once into scratch before
their rows are copied: bit for bit against the oracle, and under CUDA graphs
whose scratch no later call may take away."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import fp8_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dg():
    import precision_matmul_dg_gb300 as m
    m.lib()
    return m


def case(dg, tokens, top_k, count, width, align, dtype, seed, bad=0.05):
    """x on the GPU, its row_slot with dropped choices, and the expected codes and scales."""
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, count, (tokens, top_k)).astype(np.int32)
    ids[rng.random(ids.shape) < bad] = -1
    rows = dg.moe_rows(tokens, top_k, count, align)
    ld = (width + 7) // 8 * 8 + 8
    x = (torch.from_numpy(rng.normal(size=(tokens, ld))) *
         torch.from_numpy(np.exp2(rng.integers(-6, 7, (tokens, 1))))).to(TYPES[dtype])
    slots = torch.from_numpy(ref.sort_by_expert(ids, count, align, rows)[1])
    return x.cuda()[:, :width], slots.cuda(), x[:, :width].double().numpy(), slots.numpy()


def expected(x64, slots, top_k):
    # a row's codes and scales are its token's: quantized once, with a row of zeros last
    codes, scales = ref.quantize(np.concatenate([x64, np.zeros((1, x64.shape[1]))]))
    token = np.where(slots >= 0, slots // top_k, len(x64))
    return codes[token], scales[token]


def outputs(rows, width, pad=16, fill=0x55):
    room = torch.full((rows, (width + 15) // 16 * 16 + pad), fill, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, -(-width // 128) + 1), -3.0, device="cuda")
    return room, scales, room.view(F8)[:, :width], scales[:, :-1]


def same(codes, scales, want):
    got = codes.contiguous().view(torch.uint8).cpu().numpy()
    return np.array_equal(ref.VALUES[got], ref.VALUES[want[0]]) and \
        np.array_equal(scales.cpu().numpy(), want[1])


@pytest.mark.parametrize("tokens,top_k,count,width,align,dtype", [
    (640, 8, 16, 2057, 1, "f16"),     # odd: the last 16 bytes of a row are cut
    (700, 8, 20, 2048, 128, "bf16"),  # whole lines
    (2500, 4, 64, 1001, 1, "bf16"),   # a part-filled last block, most lanes one piece
    (90000, 2, 3, 60, 1, "f16"),      # less than a block
    (8, 8, 64, 2049, 128, "f16"),     # few tokens, mostly padding rows
])
def test_dispatch_by_way_of_scratch(dg, tokens, top_k, count, width, align, dtype):
    x, row_slot, x64, slots = case(dg, tokens, top_k, count, width, align, dtype, tokens + width)
    rows = len(slots)
    assert dg.lib().dg_moe_dispatch_fp8_scratch(tokens, top_k, width, rows) > 0
    room, wide, codes, scales = outputs(rows, width)
    before = dg.launch_count()
    dg.moe_dispatch_fp8(x, row_slot, top_k, codes, scales)
    dg.check_status()
    assert dg.launch_count() - before == 2
    assert same(codes, scales, expected(x64, slots, top_k))
    assert (room[:, width:] == 0x55).all() and (wide[:, -1] == -3.0).all()
    # without scratch: one launch, the same bits
    room2, wide2, codes2, scales2 = outputs(rows, width)
    st = dg.lib().dg_moe_dispatch_fp8(
        tokens, top_k, width, dg.F16 if dtype == "f16" else dg.BF16, x.data_ptr(), x.stride(0),
        rows, row_slot.data_ptr(), codes2.data_ptr(), codes2.stride(0), scales2.data_ptr(),
        scales2.stride(0), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0, dg.last_error()
    assert torch.equal(room, room2) and torch.equal(wide, wide2)


def test_scratch_is_left_alone_past_its_size(dg):
    tokens, top_k, width = 600, 8, 2057
    x, row_slot, x64, slots = case(dg, tokens, top_k, 16, width, 1, "f16", 4)
    rows = len(slots)
    need = dg.lib().dg_moe_dispatch_fp8_scratch(tokens, top_k, width, rows)
    scratch = torch.full((need + 64,), 0x11, dtype=torch.uint8, device="cuda")
    _, _, codes, scales = outputs(rows, width)
    st = dg.lib().dg_moe_dispatch_fp8_ex(
        tokens, top_k, width, dg.F16, x.data_ptr(), x.stride(0), rows, row_slot.data_ptr(),
        codes.data_ptr(), codes.stride(0), scales.data_ptr(), scales.stride(0), scratch.data_ptr(),
        need, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0, dg.last_error()
    assert same(codes, scales, expected(x64, slots, top_k))
    assert (scratch[need:] == 0x11).all()


def test_graph_keeps_its_scratch(dg):
    """Captured, then a larger call and a widened product on the same stream
    (either grows what the library keeps for it), then replayed on new values:
    on the capturing stream and, two graphs at once, on others."""
    tokens, top_k, width = 640, 8, 2057
    stream = torch.cuda.Stream()
    runs = []
    for seed in (1, 2):
        x, row_slot, _, _ = case(dg, tokens, top_k, 16, width, 1, "bf16", seed)
        _, _, codes, scales = outputs(row_slot.shape[0], width)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            dg.moe_dispatch_fp8(x, row_slot, top_k, codes, scales)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            dg.moe_dispatch_fp8(x, row_slot, top_k, codes, scales)
        runs.append((graph, x, row_slot, codes, scales))
    with torch.cuda.stream(stream):
        big, big_slot, big64, big_slots = case(dg, 3000, top_k, 16, width, 1, "bf16", 9)
        _, _, bc, bs = outputs(len(big_slots), width)
        dg.moe_dispatch_fp8(big, big_slot, top_k, bc, bs)
        a = torch.ones(4096, 4096, dtype=torch.int8, device="cuda")
        c = torch.zeros(4096, 4096, dtype=torch.int32, device="cuda")
        dg.gemm(a, a, c)
        # what a freed buffer would be given to
        junk = [torch.full((4 << 20,), 0x33, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert same(bc, bs, expected(big64, big_slots, top_k)) and (c == 4096).all()
    for others in ((stream, stream), (torch.cuda.Stream(), torch.cuda.Stream())):
        wants = []
        for i, (graph, x, row_slot, codes, scales) in enumerate(runs):
            nx, nslot, nx64, nslots = case(dg, tokens, top_k, 16, width, 1, "bf16", 20 + i)
            x.copy_(nx)
            row_slot.copy_(nslot)
            codes.view(torch.uint8).fill_(0)
            wants.append(expected(nx64, nslots, top_k))
        torch.cuda.synchronize()
        for s, run in zip(others, runs):
            with torch.cuda.stream(s):
                run[0].replay()
        torch.cuda.synchronize()
        for run, want in zip(runs, wants):
            assert same(run[3], run[4], want)
    assert all((j == 0x33).all() for j in junk)


@pytest.mark.parametrize("how", ["stream", "handle", "default"])
def test_dispatch_on_a_given_stream(dg, how):
    tokens, top_k, width = 640, 8, 2048
    x, row_slot, x64, slots = case(dg, tokens, top_k, 16, width, 1, "f16", 3)
    _, _, codes, scales = outputs(len(slots), width)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    dg.moe_dispatch_fp8(x, row_slot, top_k, codes, scales,
                        stream={"stream": s, "handle": s.cuda_stream, "default": 0}[how])
    torch.cuda.synchronize()
    assert same(codes, scales, expected(x64, slots, top_k))
