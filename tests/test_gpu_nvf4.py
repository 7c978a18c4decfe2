"""NVF4 (E2M1 codes, an E4M3 scale per 16 values, an FP32 scale per row):
quantization bit for bit, reading back exactly, products within the bound that
oracle.nvf4_ref derives for FP32 sums and one rounding."""

import numpy as np
import pytest
import torch

from oracle import fp8_ref, nvf4_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dg():
    import precision_matmul_dg_gb300 as m
    m.lib()
    return m


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rows16(rows, cols, seed, dtype="f16", pad=8):
    """Normal rows with their own magnitudes on the GPU, in a wider buffer, and as float64."""
    g = torch.Generator().manual_seed(seed)
    ld = (cols + 7) // 8 * 8 + pad
    x = torch.randn(rows, ld, generator=g) * torch.exp2(
        torch.randint(-6, 7, (rows, 1), generator=g).float())
    x = x.to(TYPES[dtype])
    return x.cuda()[:, :cols], x[:, :cols].double().numpy()


def buffers(rows, K, fill=0x55, pad=16):
    """Output buffers full of a pattern, with room past each row of codes."""
    ld = (K + 31) // 32 * 16 + pad
    room = torch.full((rows, ld), fill, dtype=torch.uint8, device="cuda")
    scales = torch.full((-(-rows // 128), -(-K // 64), 32, 16), fill, dtype=torch.uint8,
                        device="cuda")
    return room, (room[:, :(K + 1) // 2], scales.view(torch.float8_e4m3fn),
                  torch.full((rows,), -3.0, device="cuda"))


def same(out, want):
    """Whether (codes, scales, row scales) on the GPU are the oracle's."""
    codes, scales, rows = want
    return (np.array_equal(out[0].cpu().numpy(), ref.pack(codes)) and
            np.array_equal(out[1].view(torch.uint8).cpu().numpy(), ref.tiles(scales)) and
            np.array_equal(out[2].cpu().numpy(), rows, equal_nan=True))


def operand(rows, K, seed, scale=1.0, pad=0):
    """An operand on the GPU (garbage past the rows' codes), and its values in 64 bits."""
    rng = np.random.default_rng(seed)
    codes, scales, r = ref.quantize(rng.normal(size=(rows, K)) * scale *
                                    np.exp2(rng.integers(-3, 4, (rows, 1))))
    r = (r * rng.uniform(0.6, 1.7, rows)).astype(np.float32)
    room = np.full((rows, (K + 31) // 32 * 16 + pad), 0x77, np.uint8)
    room[:, :(K + 1) // 2] = ref.pack(codes)
    return ((gpu(room)[:, :(K + 1) // 2], gpu(ref.tiles(scales)).view(torch.float8_e4m3fn), gpu(r)),
            ref.values(codes, scales, r))


def check(got, t, err, dtype):
    g = got.double().cpu().numpy()
    bound = fp8_ref.rounded_bound(t, err, dtype)
    bad = ~(np.abs(g - t) <= bound)
    assert not bad.any(), "%d of %d outside the bound, first at %s: %r for %r, bound %r" % (
        bad.sum(), bad.size, np.argwhere(bad)[0], g[bad][0], t[bad][0], bound[bad][0])


# --------------------------------------------------------------- quantization

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 16), (3, 127), (16, 4096), (129, 257), (130, 1000),
                                    (5, 63), (300, 40), (2, 17000), (31, 8200)])
def test_quantize(dg, rows, K, dtype):
    x, x64 = rows16(rows, K, rows * 7 + K, dtype)
    room, out = buffers(rows, K)
    got = dg.quantize_nvf4(x, out=out)
    dg.check_status()
    want = ref.quantize(x64)
    assert same(got, want)
    assert (room[:, (K + 1) // 2:] == 0x55).all()
    for t in ("f16", "bf16", "f32"):
        wide = torch.full((rows, K + 3), 7.0, dtype=TYPES[t], device="cuda")
        d = dg.dequantize_nvf4(*got, wide[:, :K])
        v = torch.from_numpy(ref.values(*want)).float().to(TYPES[t])
        assert torch.equal(d.cpu(), v) and (wide[:, K:] == 7.0).all()
        aligned = dg.dequantize_nvf4(*got, torch.empty(rows, (K + 7) // 8 * 8, dtype=TYPES[t],
                                                       device="cuda")[:, :K])
        assert torch.equal(aligned.cpu(), v)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_quantize_special_values(dg, dtype):
    x64 = np.random.default_rng(5).normal(size=(130, 300))
    x64[0, 3], x64[1, 200], x64[2, 299] = np.inf, np.nan, -np.inf
    x64[3] = 0.0
    x64[4, :128] = 0.0
    x64[5] = 2.0 ** -24
    x64[6, 7] = 60000.0
    x64[7] = -0.0
    x64[8] = np.nan
    x64[9, ::2] = -1e-5
    x = torch.from_numpy(x64).to(TYPES[dtype])
    room = torch.zeros(130, 304, dtype=x.dtype)
    room[:, :300] = x
    got = dg.quantize_nvf4(room.cuda()[:, :300])
    want = ref.quantize(x.double().numpy())
    assert same(got, want)
    d = dg.dequantize_nvf4(*got, torch.empty(130, 300, device="cuda"))
    assert np.array_equal(d.double().cpu().numpy(), ref.values(*want), equal_nan=True)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_quantize_every_largest_value(dg, dtype):
    # a row for every finite magnitude, as the only value and beside others
    bits = np.arange(0, 0x7C00 if dtype == "f16" else 0x7F80, 3).astype(np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).view(TYPES[dtype])
    rows = torch.zeros(len(bits), 32, dtype=x.dtype)
    rows[:, 5] = x
    rows[:, 20] = -x * 0.7
    assert same(dg.quantize_nvf4(rows.cuda()), ref.quantize(rows.double().numpy()))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_quantize_middles(dg, dtype):
    # values in the middle between two codes, and one step beside it, for every scale
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    rows = np.zeros((126, 64))
    for s in range(1, 127):
        v = mids * fp8_ref.VALUES[s]
        rows[s - 1, :8], rows[s - 1, 8:16] = v, -v
        rows[s - 1, 16:24] = v * (1 + 2.0 ** -7)
        rows[s - 1, 24:32] = v * (1 - 2.0 ** -7)
    rows[:, 48] = 2688.0  # the row's scale is 1
    x = torch.from_numpy(rows).to(TYPES[dtype])
    assert same(dg.quantize_nvf4(x.cuda()), ref.quantize(x.double().numpy()))


def test_quantize_with_given_row_scales(dg):
    x, x64 = rows16(140, 100, 3, "bf16")
    rng = np.random.default_rng(4)
    given = (np.exp2(rng.uniform(-16, 4, 140))).astype(np.float32)
    given[:8] = [0.0, np.nan, np.inf, -1.0, 2.0 ** -101, 2.0 ** 101, 2.0 ** -100, 2.0 ** 100]
    got = dg.quantize_nvf4(x, row_scales=gpu(given))
    assert same(got, ref.quantize(x64, given))
    room, out = buffers(140, 100)
    got = dg.quantize_nvf4(x, row_scales=gpu(given), out=(out[0], out[1], None))
    assert same(got, ref.quantize(x64, given))
    big = torch.full((1, 32), 3e38, dtype=torch.bfloat16, device="cuda")
    small = gpu(np.array([2.0 ** -100], np.float32))
    assert same(dg.quantize_nvf4(big, row_scales=small),
                ref.quantize(big.double().cpu().numpy(), small.cpu().numpy()))


@pytest.mark.parametrize("count,rows,K", [(3, 130, 70), (5, 1, 33), (2, 256, 512)])
def test_stack(dg, count, rows, K):
    x, x64 = rows16(count * rows, K, 11, "f16")
    got = dg.quantize_nvf4(x.unflatten(0, (count, rows)))
    d = dg.dequantize_nvf4(*got, torch.empty(count, rows, K, device="cuda"))
    for z in range(count):
        want = ref.quantize(x64[z * rows:(z + 1) * rows])
        assert same([t[z] for t in got], want)
        assert np.array_equal(d[z].double().cpu().numpy(), ref.values(*want))


@pytest.mark.parametrize("align", [1, 128])
def test_dispatch(dg, align):
    tokens, top_k, count, width = 40, 3, 6, 200
    rng = np.random.default_rng(2)
    x, x64 = rows16(tokens, width, 1, "bf16")
    ids = rng.integers(-1, count + 1, (tokens, top_k)).astype(np.int32)
    rows = dg.moe_rows(tokens, top_k, count, align)
    _, row_slot, _ = fp8_ref.sort_by_expert(ids, count, align, rows)
    row_slot[-1] = tokens * top_k  # a token past the last: zeros
    room, out = buffers(rows, width)
    dg.moe_dispatch_nvf4(x, gpu(row_slot), top_k, *out)
    want = fp8_ref.dispatch(np.concatenate([x64, np.zeros((1, width))]), row_slot, top_k)
    assert same(out, ref.quantize(want)) and (room[:, 100:] == 0x55).all()


# -------------------------------------------------------------------- product

SHAPES = [(1, 1, 1), (1, 64, 64), (3, 200, 16), (17, 300, 1000), (128, 128, 256), (130, 70, 333),
          (128, 192, 64), (300, 500, 520), (512, 400, 2048), (257, 1000, 777), (1000, 193, 130),
          (64, 4100, 300), (5, 129, 4096)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(dg, M, N, K):
    a, av = operand(M, K, 1 + M, pad=16)
    b, bv = operand(N, K, 2 + N)
    t, err = ref.product(av, bv)
    for dtype in ("f16", "bf16", "f32"):
        wide = torch.full((M, N + 5), 3.0, dtype=TYPES[dtype], device="cuda")
        check(dg.gemm_nvf4(*a, *b, wide[:, :N]), t, err, dtype)
        assert (wide[:, N:] == 3.0).all()
        aligned = torch.zeros(M, (N + 7) // 8 * 8, dtype=TYPES[dtype], device="cuda")[:, :N]
        check(dg.gemm_nvf4(*a, *b, aligned), t, err, dtype)
        assert torch.equal(aligned, wide[:, :N])
    dg.check_status()


@pytest.mark.parametrize("M", [9, 200, 300])
@pytest.mark.parametrize("epilogue", ["none", "bias", "gelu", "bias_gelu"])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_epilogues(dg, M, epilogue, dtype):
    N, K = 456, 640
    a, av = operand(M, K, 5)
    b, bv = operand(N, K, 6, scale=K ** -0.5)
    rng = np.random.default_rng(7)
    d = torch.from_numpy(rng.normal(size=(M, N))).to(TYPES[dtype])
    bias = torch.from_numpy(rng.normal(size=N)).to(TYPES[dtype])
    t, err = ref.product(av, bv, -0.75, 0.5, d.double().numpy(),
                         bias.double().numpy() if "bias" in epilogue else None, "gelu" in epilogue)
    got = dg.gemm_nvf4(*a, *b, d.cuda(), bias=bias.cuda(), alpha=-0.75, beta=0.5,
                       epilogue=epilogue)
    check(got, t, err, dtype)


def test_gemm_nan_scales_stay_in_their_row(dg):
    a, av = operand(300, 300, 8)
    b, bv = operand(260, 300, 9)
    a[1].view(torch.uint8)[1, 2, 5, 1] = 0x7F   # row 133, block 9
    b[1].view(torch.uint8)[0, 0, 31, 12] = 0x7F  # row 127, block 0
    t, err = ref.product(av, bv)
    d = dg.gemm_nvf4(*a, *b, torch.zeros(300, 260, device="cuda"))
    nan = torch.isnan(d)
    assert nan[133].all() and nan[:, 127].all() and nan.sum() == 300 + 260 - 1
    keep = ~nan.cpu().numpy()
    assert (np.abs(d.double().cpu().numpy() - t) <= fp8_ref.rounded_bound(t, err, "f32"))[keep].all()


def test_gemm_does_not_read_scales_past_k(dg):
    # the last scale tile's neighbours are NaN: the next rows' tiles and what follows the last
    K = 320  # 5 tiles: a stage and a quarter
    a, av = operand(128, K, 10)
    b, bv = operand(192, K, 11)
    ops = []
    for codes, scales, rows in (a, b):
        room = torch.full((scales.numel() + 8 * 512,), 0x7F, dtype=torch.uint8, device="cuda")
        room[:scales.numel()] = scales.view(torch.uint8).reshape(-1)
        ops.append((codes, room[:scales.numel()].view(torch.float8_e4m3fn).reshape(scales.shape), rows))
    t, err = ref.product(av, bv)
    for m in (128, 40):
        first = tuple(v[:m] if i != 1 else v for i, v in enumerate(ops[0]))
        check(dg.gemm_nvf4(*first, *ops[1], torch.zeros(m, 192, device="cuda")), t[:m], err[:m],
              "f32")


def grouped_case(dg, sizes, N, K, seed, extra=0):
    count = len(sizes)
    ends = np.cumsum([0] + [-(-s // 128) * 128 for s in sizes])
    rows = int(ends[-1]) + extra
    a, av = operand(rows, K, seed)
    parts = [operand(N, K, seed + 1 + e, scale=K ** -0.5) for e in range(count)]
    b = tuple(torch.stack([p[0][i].view(torch.uint8) if i == 1 else p[0][i] for p in parts])
              for i in range(3))
    ld = -(-K // 32) * 16
    room = torch.full((count, N + 3, ld), 0x33, dtype=torch.uint8, device="cuda")
    room[:, :N, :(K + 1) // 2] = b[0]
    b = (room[:, :N, :(K + 1) // 2], b[1].view(torch.float8_e4m3fn).contiguous(), b[2].contiguous())
    return a, av, b, [p[1] for p in parts], gpu(ends.astype(np.int32)), ends


@pytest.mark.parametrize("sizes,N,K", [([5, 0, 130, 300], 200, 300), ([1], 70, 64),
                                       ([600, 700, 0, 129], 400, 512), ([0, 0], 64, 64),
                                       ([256, 1, 1, 1, 1, 1, 1, 900], 136, 1100)])
def test_grouped(dg, sizes, N, K):
    a, av, b, bv, offsets, ends = grouped_case(dg, sizes, N, K, 20, extra=128)
    rng = np.random.default_rng(21)
    bias = torch.from_numpy(rng.normal(size=(len(sizes), N))).float()
    for dtype, epilogue in (("bf16", "none"), ("f32", "bias_gelu")):
        d = torch.full((len(av), N), 9.0, dtype=TYPES[dtype], device="cuda")
        dg.gemm_nvf4_grouped(*a, *b, offsets, d, bias=bias.to(TYPES[dtype]).cuda(),
                             epilogue=epilogue)
        dg.check_status()
        for e in range(len(sizes)):
            at = slice(ends[e], ends[e + 1])
            t, err = ref.product(av[at], bv[e],
                                 bias=bias[e].double().numpy() if "bias" in epilogue else None,
                                 use_gelu="gelu" in epilogue)
            check(d[at], t, err, dtype)
        assert (d[ends[-1]:] == 9.0).all()


def test_grouped_offsets(dg):
    # clamped to the rows; an end before its start is empty; off a tile: rounded down and reported
    a, av, b, bv, _, _ = grouped_case(dg, [128, 128, 128], 96, 128, 30)
    for off, segments, status in (([0, 128, 128, 5000], [(0, 128), (128, 128), (128, 384)], None),
                                  ([-5, 256, 128, 384], [(0, 256), (256, 256), (128, 384)], None),
                                  ([0, 130, 256, 384], [(0, 128), (128, 256), (256, 384)], 1)):
        d = torch.full((384, 96), 9.0, device="cuda")
        dg.gemm_nvf4_grouped(*a, *b, gpu(np.array(off, np.int32)), d)
        if status is None:
            dg.check_status()
        else:
            with pytest.raises(dg.DgError, match="status word %d" % status):
                dg.check_status()
        # (the second list's segments overlap in rows 128 .. 255: either expert's)
        for e, (lo, hi) in enumerate(segments):
            lo = 256 if off[0] < 0 and e == 2 else lo
            if off[0] < 0 and e == 0:
                hi = 128
            if hi > lo:
                t, err = ref.product(av[lo:hi], bv[e])
                check(d[lo:hi], t, err, "f32")


def test_graph_and_streams(dg):
    x, _ = rows16(300, 512, 40, "bf16")
    b, bv = operand(200, 512, 41)
    s = torch.cuda.Stream()
    out = dg.nvf4_buffers(300, 512)
    d = torch.empty(300, 200, device="cuda")

    def step():
        dg.quantize_nvf4(x, out=out)
        dg.gemm_nvf4(*out, *b, d)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    x2, x64 = rows16(300, 512, 42, "bf16")
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    want = ref.quantize(x64)
    assert same(out, want)
    t, err = ref.product(ref.values(*want), bv)
    check(d, t, err, "f32")
    d.zero_()
    torch.cuda.synchronize()
    dg.gemm_nvf4(*out, *b, d, stream=s)
    s.synchronize()
    check(d, t, err, "f32")


# ------------------------------------- enough tiles for pairs of 256 x 192
@pytest.mark.parametrize("M,N,K,dtype,epilogue", [(1000, 2900, 200, "bf16", "none"),
                                                  (1024, 2880, 256, "f16", "bias"),
                                                  (1025, 2881, 777, "f32", "bias_gelu"),
                                                  (897, 2913, 64, "bf16", "bias_gelu"),
                                                  (2100, 1500, 1, "f16", "none")])
def test_pairs(dg, M, N, K, dtype, epilogue):
    a, av = operand(M, K, 60, pad=16)
    b, bv = operand(N, K, 61, scale=K ** -0.5)
    rng = np.random.default_rng(62)
    d = torch.from_numpy(rng.normal(size=(M, N))).to(TYPES[dtype])
    bias = torch.from_numpy(rng.normal(size=N)).to(TYPES[dtype])
    t, err = ref.product(av, bv, 1.25, -0.5, d.double().numpy(),
                         bias.double().numpy() if "bias" in epilogue else None, "gelu" in epilogue)
    wide = torch.full((M + 3, N + 5), 3.0, dtype=TYPES[dtype], device="cuda")
    wide[:M, :N] = d.cuda()
    check(dg.gemm_nvf4(*a, *b, wide[:M, :N], bias=bias.cuda(), alpha=1.25, beta=-0.5,
                       epilogue=epilogue), t, err, dtype)
    assert (wide[:, N:] == 3.0).all() and (wide[M:] == 3.0).all()
    aligned = torch.empty(M, (N + 7) // 8 * 8, dtype=TYPES[dtype], device="cuda")[:, :N]
    aligned.copy_(d)
    dg.gemm_nvf4(*a, *b, aligned, bias=bias.cuda(), alpha=1.25, beta=-0.5, epilogue=epilogue)
    assert torch.equal(aligned, wide[:M, :N])
    dg.check_status()


def test_pairs_nan_scales_stay_in_their_row(dg):
    M, N, K = 1000, 2900, 320  # K: five scale tiles, and NaN behind the last
    a, av = operand(M, K, 63)
    b, bv = operand(N, K, 64)
    room = torch.full((b[1].numel() + 4096,), 0x7F, dtype=torch.uint8, device="cuda")
    room[:b[1].numel()] = b[1].view(torch.uint8).reshape(-1)
    b = (b[0], room[:b[1].numel()].view(torch.float8_e4m3fn).reshape(b[1].shape), b[2])
    a[1].view(torch.uint8)[3, 2, 5, 1] = 0x7F  # row 389, block 9
    b[1].view(torch.uint8)[22, 0, 31, 4] = 0x7F  # row 2879, block 0
    t, err = ref.product(av, bv)
    d = dg.gemm_nvf4(*a, *b, torch.zeros(M, N, device="cuda"))
    nan = torch.isnan(d)
    assert nan[389].all() and nan[:, 2879].all() and nan.sum() == M + N - 1
    keep = ~nan.cpu().numpy()
    assert (np.abs(d.double().cpu().numpy() - t) <= fp8_ref.rounded_bound(t, err, "f32"))[keep].all()


@pytest.mark.parametrize("sizes,N,K", [([600, 700, 900], 200, 300), ([1, 1500, 0, 900], 400, 512),
                                       ([129, 2000], 392, 64)])
def test_grouped_pairs(dg, sizes, N, K):
    test_grouped(dg, sizes, N, K)


def test_grouped_pairs_of_many_experts(dg):
    # more experts than a fifth stage leaves room for, and most of the rows in none
    count, N, K = 250, 40, 48
    rng = np.random.default_rng(65)
    sizes = rng.integers(0, 3, count) * 128
    ends = np.cumsum(np.concatenate([[0], sizes]))
    rows = 512 * count
    a, av = operand(rows, K, 66)
    b, bv = operand(count * N, K, 67)
    b3 = (b[0].reshape(count, N, -1).contiguous(),
          gpu(np.stack([ref.tiles(s) for s in untiled(b[1], count * N, K).reshape(count, N, -1)])),
          b[2].reshape(count, N))
    room = torch.zeros(count, N, 32, dtype=torch.uint8, device="cuda")
    room[:, :, :K // 2] = b3[0]
    d = torch.full((rows, N), 9.0, device="cuda")
    dg.gemm_nvf4_grouped(*a, room[:, :, :K // 2], b3[1].view(torch.float8_e4m3fn), b3[2],
                         gpu(ends.astype(np.int32)), d)
    dg.check_status()
    bv = bv.reshape(count, N, K)
    for e in range(count):
        at = slice(ends[e], ends[e + 1])
        if ends[e + 1] > ends[e]:
            t, err = ref.product(av[at], bv[e])
            check(d[at], t, err, "f32")
    assert (d[ends[-1]:] == 9.0).all()


def untiled(scales, rows, K):
    """The scale codes [rows, blocks] of tiles (numpy)."""
    t = scales.view(torch.uint8).cpu().numpy()
    m, k = t.shape[:2]
    full = t.reshape(m, k, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(m * 128, k * 4)
    return full[:rows, :-(-K // 16)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("offset,pitch", [(0, 104), (1, 104), (0, 101), (3, 107)])
def test_reading_back_into_any_rows(dg, dtype, offset, pitch):
    rows, K = 131, 100
    (codes, scales, r), _ = operand(rows, K, 68)
    # the formula's steps, each rounded to FP32: code * (scale * row scale)
    one = np.ones(rows, np.float32)
    packed = codes.cpu().numpy()
    plain = np.stack([packed & 15, packed >> 4], -1).reshape(rows, K)
    of_block = untiled(scales, rows, K)
    code = ref.values(plain, np.full_like(of_block, 0x38), one).astype(np.float32)
    scale = ref.values(np.full_like(plain, 2), of_block, one).astype(np.float32)
    v = code * (scale * r.cpu().numpy()[:, None])
    assert v.dtype == np.float32
    room = torch.full((rows * pitch + 8,), 7.0, dtype=TYPES[dtype], device="cuda")
    d = room[offset:].as_strided((rows, K), (pitch, 1), room.storage_offset() + offset)
    dg.dequantize_nvf4(codes, scales, r, d)
    assert torch.equal(d.cpu(), torch.from_numpy(v).to(TYPES[dtype]))
    outside = torch.ones(rows * pitch + 8, dtype=torch.bool)
    outside.as_strided((rows, K), (pitch, 1), offset)[:] = False
    assert (room.cpu()[outside] == 7.0).all()
