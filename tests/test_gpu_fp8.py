"""FP8 (E4M3 with block scales): quantization bit for bit, products within the
bound that oracle.fp8_ref derives for FP32 sums and one rounding."""

import numpy as np
import pytest
import torch

from oracle import fp8_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dg():
    import precision_matmul_dg_gb300 as m
    m.lib()
    return m


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rows16(rows, cols, seed, dtype="f16", scale=1.0, pad=8):
    """Normal rows with their own magnitudes on the GPU, in a wider buffer, and as float64."""
    g = torch.Generator().manual_seed(seed)
    ld = (cols + 7) // 8 * 8 + pad
    x = torch.randn(rows, ld, generator=g) * torch.exp2(
        torch.randint(-6, 7, (rows, 1), generator=g).float()) * scale
    x = x.to(TYPES[dtype])
    return x.cuda()[:, :cols], x[:, :cols].double().numpy()


def codes_of(t):
    return t.cpu().contiguous().view(torch.uint8).numpy()


def operand(rows, K, seed, block_rows=1, scale=1.0, pad=0):
    """E4M3 codes (pitch a multiple of 16 plus pad, NaN codes past K) with scales on the GPU,
    and their values in 64 bits."""
    rng = np.random.default_rng(seed)
    codes, scales = ref.quantize(rng.normal(size=(rows, K)) * scale, block_rows)
    ld = (K + 15) // 16 * 16 + pad
    room = np.full((rows, ld), 0x7F, np.uint8)
    room[:, :K] = codes
    return (gpu(room).view(torch.float8_e4m3fn)[:, :K], gpu(scales),
            ref.values(codes, scales, block_rows))


# --------------------------------------------------------------- quantization

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 128), (3, 127), (16, 4096), (129, 257), (200, 1000),
                                    (256, 128), (31, 16)])
def test_quantize(dg, rows, K, block_rows, dtype):
    x, x64 = rows16(rows, K, rows * 7 + K, dtype)
    want = ref.quantize(x64, block_rows) + ref.quantize(x64.T, block_rows)
    for form, pick in (("rows", (0, 1)), ("transposed", (2, 3)), ("both", (0, 1, 2, 3))):
        got = dg.quantize_fp8(x, form=form, block_rows=block_rows)
        for i, k in enumerate(pick):
            g = codes_of(got[i]) if k % 2 == 0 else got[i].cpu().numpy()
            assert np.array_equal(g, want[k]), (form, k)
    dg.check_status()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_quantize_special_values(dg, dtype):
    x64 = np.random.default_rng(5).normal(size=(130, 300))
    x64[0, 3], x64[1, 200], x64[2, 299] = np.inf, np.nan, -np.inf
    x64[3] = 0.0
    x64[4, :128] = 0.0
    x64[5] = 2.0 ** -24
    x64[6, 7] = 60000.0
    x64[7] = -0.0
    x = torch.from_numpy(x64).to(TYPES[dtype])
    room = torch.zeros(130, 304, dtype=x.dtype)
    room[:, :300] = x
    xg = room.cuda()[:, :300]
    for br in (1, 128):
        want = ref.quantize(x.double().numpy(), br) + ref.quantize(x.double().numpy().T, br)
        got = dg.quantize_fp8(xg, form="both", block_rows=br)
        for i in (0, 2):
            assert np.array_equal(ref.VALUES[codes_of(got[i])], ref.VALUES[want[i]])
        for i in (1, 3):
            assert np.array_equal(got[i].cpu().numpy(), want[i], equal_nan=True)
        row = dg.quantize_fp8(xg, block_rows=br)
        assert np.array_equal(codes_of(row[0]), codes_of(got[0]))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_quantize_every_largest_value(dg, dtype):
    # a block for every finite magnitude: scales and factors are the rounded quotients
    bits = np.arange(0, 0x7C00 if dtype == "f16" else 0x7F80).astype(np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).view(TYPES[dtype])
    rows = torch.zeros(len(bits), 128, dtype=x.dtype)
    rows[:, 5] = x
    rows[:, 77] = -x * 0.7
    got = dg.quantize_fp8(rows.cuda())
    want = ref.quantize(rows.double().numpy())
    assert np.array_equal(got[1].cpu().numpy(), want[1])
    assert np.array_equal(ref.VALUES[codes_of(got[0])], ref.VALUES[want[0]])


def test_quantize_smallest_bf16(dg):
    x = torch.full((2, 128), 1e-39, dtype=torch.bfloat16)
    x[1] = 3e38
    want = ref.quantize(x.double().numpy())
    got = dg.quantize_fp8(x.cuda())
    assert np.array_equal(codes_of(got[0]), want[0])
    assert np.array_equal(got[1].cpu().numpy(), want[1])


def test_quantize_leaves_the_padding(dg):
    rows, K = 37, 200
    x, _ = rows16(rows, K, 9)
    rooms = [torch.full((rows, 224), 0x55, dtype=torch.uint8, device="cuda"),
             torch.full((K, 64), 0x55, dtype=torch.uint8, device="cuda")]
    s = [torch.full((rows, 5), -3.0, device="cuda"), torch.full((K, 3), -3.0, device="cuda")]
    f8 = [r.view(torch.float8_e4m3fn) for r in rooms]
    dg.quantize_fp8(x, form="both", out=(f8[0][:, :K], s[0][:, :2], f8[1][:, :rows], s[1][:, :1]))
    assert (rooms[0][:, K:] == 0x55).all() and (rooms[1][:, rows:] == 0x55).all()
    assert (s[0][:, 2:] == -3.0).all() and (s[1][:, 1:] == -3.0).all()
    rooms[0].fill_(0x55)
    dg.quantize_fp8(x, out=(f8[0][:, :K], s[0][:, :2]))
    assert (rooms[0][:, K:] == 0x55).all()


# -------------------------------------------------------------------- product

def check(got, t, err, dtype):
    g = got.double().cpu().numpy()
    bound = ref.rounded_bound(t, err, dtype)
    bad = ~(np.abs(g - t) <= bound)
    assert not bad.any(), "%d of %d outside the bound, first at %s: %r for %r, bound %r" % (
        bad.sum(), bad.size, np.argwhere(bad)[0], g[bad][0], t[bad][0], bound[bad][0])


SIZES = [(1, 1, 1), (1, 8960, 1536), (3, 100, 128), (8, 256, 129), (9, 31, 700), (16, 513, 2064),
         (17, 64, 128), (31, 130, 127), (100, 200, 1000), (128, 256, 512), (129, 257, 640),
         (300, 1000, 384), (257, 520, 2049), (1024, 1100, 256), (2100, 2300, 300), (777, 7000, 130),
         (2048, 2560, 1152),
         (65, 300, 2049), (200, 130, 4100), (70, 1000, 6000), (130, 515, 8200), (300, 1000, 2900)]


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gemm(dg, M, N, K, block_rows):
    a, sa, av = operand(M, K, M + K, pad=16)
    b, sb, bv = operand(N, K, N + K + 1, block_rows, scale=0.05)
    for dtype in ("f16", "bf16", "f32"):
        d = torch.full((M, N), float("nan"), dtype=TYPES[dtype], device="cuda")
        dg.gemm_fp8(a, sa, b, sb, d)
        dg.check_status()
        check(d, *ref.product(av, bv), dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(5, 300, 256), (150, 300, 400)])
@pytest.mark.parametrize("epilogue", ["none", "bias", "gelu", "bias_gelu"])
def test_gemm_epilogue(dg, M, N, K, dtype, epilogue):
    a, sa, av = operand(M, K, 1)
    b, sb, bv = operand(N, K, 2, 128, scale=0.05)
    t = TYPES[dtype]
    bias = torch.randn(N, generator=torch.Generator().manual_seed(3)).to(t)
    room = torch.randn(M, N + 5, generator=torch.Generator().manual_seed(4)).to(t).cuda()
    before = room.clone()
    d = room[:, :N]
    args = dict(alpha=0.75, beta=-0.5, d=before[:, :N].double().cpu().numpy(),
                use_gelu="gelu" in epilogue,
                bias=bias.double().numpy() if "bias" in epilogue else None)
    dg.gemm_fp8(a, sa, b, sb, d, bias=bias.cuda(), alpha=0.75, beta=-0.5, epilogue=epilogue)
    dg.check_status()
    check(d, *ref.product(av, bv, **args), dtype)
    assert torch.equal(room[:, N:], before[:, N:])


@pytest.mark.parametrize("M,N", [(4, 1201), (130, 1201), (5000, 1204)])
def test_gelu_over_its_range(dg, M, N):
    """Zero operands: the bias alone is GELU's argument.  Its Phi is good to
    1e-7 and the exponential's 2^-22 of at most 1/2, the result is rounded."""
    a = torch.zeros(M, 128, device="cuda").to(torch.float8_e4m3fn)
    b = torch.zeros(N, 128, device="cuda").to(torch.float8_e4m3fn)
    one = torch.ones(max(M, N), 1, device="cuda")
    t = torch.linspace(-12.0, 12.0, N)
    t[:9] = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3e4, -3e4, float("inf"), -float("inf"),
                          float("nan")])
    d = torch.empty(M, N, device="cuda")
    dg.gemm_fp8(a, one[:M], b, one[:(N + 127) // 128], d, bias=t.cuda(), epilogue="bias_gelu")
    dg.check_status()
    got = d.cpu().double()
    assert torch.equal(got.nan_to_num(-1.0), got[:1].nan_to_num(-1.0).expand_as(got))
    got = got[-1]
    assert got[6] == float("inf") and got[7] == 0.0 and torch.isnan(got[8])
    x = t.double()
    keep = torch.isfinite(x)
    want = 0.5 * x * torch.special.erfc(-x / 2.0 ** 0.5)
    bound = (1e-7 + 2.0 ** -23) * x.abs() + 2.0 ** -23 * want.abs() + 4e-12
    assert ((got - want).abs() <= bound)[keep].all()


@pytest.mark.parametrize("M", [4, 200])
def test_gemm_without_k(dg, M):
    a, sa = torch.empty(M, 0, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(M, 0).cuda()
    b, sb = torch.empty(70, 0, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(70, 0).cuda()
    d = torch.ones(M, 70, dtype=torch.float16, device="cuda")
    dg.gemm_fp8(a, sa, b, sb, d, beta=0.5)
    assert (d == 0.5).all()
    dg.gemm_fp8(a, sa, b, sb, d)
    assert (d == 0.0).all()


@pytest.mark.parametrize("M", [2, 140])
def test_gemm_scale_nan_stays_in_its_row(dg, M):
    K, N = 384, 260
    a, sa, av = operand(M, K, 11)
    b, sb, bv = operand(N, K, 12, 128, scale=0.05)
    sa[1, 1] = float("nan")
    d = torch.empty(M, N, dtype=torch.float32, device="cuda")
    dg.gemm_fp8(a, sa, b, sb, d)
    assert torch.isnan(d[1]).all()
    keep = [i for i in range(M) if i != 1]
    t, err = ref.product(av, bv)
    check(d[keep], t[keep], err[keep], "f32")


def test_gemm_is_stable_and_follows_its_stream(dg):
    a, sa, av = operand(300, 1024, 21)
    b, sb, bv = operand(500, 1024, 22, 128, scale=0.05)
    d = [torch.empty(300, 500, dtype=torch.float32, device="cuda") for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dg.gemm_fp8(a, sa, b, sb, d[0], stream=s)
    with torch.cuda.stream(s):
        dg.gemm_fp8(a, sa, b, sb, d[1])
    s.synchronize()
    assert torch.equal(d[0], d[1])
    check(d[0], *ref.product(av, bv), "f32")


# -------------------------------------------------------------------- experts

def expert_weights(count, N, K, seed):
    ld = (K + 15) // 16 * 16
    codes = np.full((count, N, ld), 0x7F, np.uint8)
    scales = np.zeros((count, -(-N // 128), -(-K // 128)), np.float32)
    values = []
    for e in range(count):
        c, scales[e] = ref.quantize(np.random.default_rng(seed + e).normal(size=(N, K)) * 0.05, 128)
        codes[e, :, :K] = c
        values.append(ref.values(c, scales[e], 128))
    return gpu(codes).view(torch.float8_e4m3fn)[:, :, :K], gpu(scales), values


GROUPS = {
    "single": [1],
    "decode": [1, 0, 2, 0, 0, 3, 1, 17],
    "empty": [0, 0, 0],
    "ragged": [130, 0, 1, 255, 64, 128],
    "one_has_all": [0, 600, 0],
    "many": [i % 5 for i in range(40)],
}


@pytest.mark.parametrize("dtype,epilogue", [("f16", "gelu"), ("bf16", "bias_gelu"), ("f32", "none")])
@pytest.mark.parametrize("N,K", [(200, 272), (513, 130), (128, 1024)])
@pytest.mark.parametrize("group", sorted(GROUPS))
def test_grouped(dg, group, N, K, dtype, epilogue):
    sizes = GROUPS[group]
    used, rows = sum(sizes), sum(sizes) + 3
    a, sa, av = operand(rows, K, 31)
    b, sb, bv = expert_weights(len(sizes), N, K, 32)
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    t = TYPES[dtype]
    bias = torch.randn(len(sizes), N, generator=torch.Generator().manual_seed(5)).to(t)
    d = torch.full((rows, N), 7.0, dtype=t, device="cuda")
    dg.gemm_fp8_grouped(a, sa, b, sb, gpu(offsets), d, bias=bias.cuda(), epilogue=epilogue)
    dg.check_status()
    assert (d[used:] == 7.0).all()
    for e in range(len(sizes)):
        at = slice(offsets[e], offsets[e + 1])
        if sizes[e]:
            check(d[at], *ref.product(av[at], bv[e], use_gelu="gelu" in epilogue,
                                      bias=bias[e].double().numpy() if "bias" in epilogue else None),
                  dtype)


def test_grouped_offsets_are_clamped(dg):
    b, sb, bv = expert_weights(3, 64, 128, 42)
    for rows in (40, 100):  # few rows per expert, and more
        a, sa, av = operand(rows, 128, 41)
        d = torch.full((rows, 64), 7.0, dtype=torch.float32, device="cuda")
        offsets = gpu(np.array([-5, 10, 4, 1000], np.int32))
        dg.gemm_fp8_grouped(a, sa, b, sb, offsets, d)
        dg.check_status()
        check(d[:4], *[x[:4] for x in ref.product(av[:4], bv[0])], "f32")
        check(d[10:], *ref.product(av[10:], bv[2]), "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N", [(64, 100), (256, 300), (129, 513), (1400, 1501)])
@pytest.mark.parametrize("sizes", [[128], [0, 256, 128, 0], [640, 128], [0]])
def test_grouped_wgrad(dg, sizes, M, N, dtype):
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    rows = int(offsets[-1]) + 128
    a, sa, av = operand(M, rows, 51)
    b, sb, bv = operand(N, rows, 52)
    d = torch.full((len(sizes), M, N + 3), 2.0, dtype=TYPES[dtype], device="cuda")
    for beta in (0.0, 0.5):
        d.fill_(2.0)
        dg.gemm_fp8_grouped_wgrad(a, sa, b, sb, gpu(offsets), d[:, :, :N], alpha=0.25, beta=beta)
        dg.check_status()
        for e in range(len(sizes)):
            at = slice(offsets[e], offsets[e + 1])
            check(d[e, :, :N], *ref.product(av[:, at], bv[:, at], alpha=0.25, beta=beta,
                                            d=np.full((M, N), 2.0)), dtype)
        assert (d[:, :, N:] == 2.0).all()


@pytest.mark.parametrize("M,N", [(600, 700), (140, 150)])
def test_grouped_wgrad_between_empty_segments(dg, M, N):
    # many empty experts at segment starts that are no multiple of four blocks,
    # several tiles to a CTA
    sizes = [0, 128, 0, 0, 384, 0] + [0, 0, 128, 0, 0] * 8 + [0] * 10
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    rows = int(offsets[-1])
    a, sa, av = operand(M, rows, 53)
    b, sb, bv = operand(N, rows, 54)
    d = torch.full((len(sizes), M, N), 2.0, device="cuda")
    dg.gemm_fp8_grouped_wgrad(a, sa, b, sb, gpu(offsets), d)
    dg.check_status()
    for e in range(len(sizes)):
        at = slice(offsets[e], offsets[e + 1])
        check(d[e], *ref.product(av[:, at], bv[:, at]), "f32")


def test_grouped_wgrad_reports_misaligned_segments(dg):
    a, sa, av = operand(32, 256, 61)
    b, sb, bv = operand(48, 256, 62)
    d = torch.zeros(2, 32, 48, device="cuda")
    dg.gemm_fp8_grouped_wgrad(a, sa, b, sb, gpu(np.array([0, 130, 256], np.int32)), d)
    with pytest.raises(dg.DgError):
        dg.check_status()
    dg.check_status()
    check(d[0], *ref.product(av[:, :128], bv[:, :128]), "f32")


def test_grouped_wgrad_without_rows(dg):
    e = torch.empty(32, 0, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(32, 0, device="cuda")
    d = torch.ones(3, 32, 32, device="cuda")
    dg.gemm_fp8_grouped_wgrad(e, s, e, s, gpu(np.zeros(4, np.int32)), d, beta=0.5)
    assert (d == 0.5).all()


# ------------------------------------------------------------------- refusals

def test_refusals(dg):
    a, sa, _ = operand(20, 256, 71)
    b, sb, _ = operand(256, 256, 72, 128)
    d = torch.zeros(20, 256, dtype=torch.float16, device="cuda")
    good = dict(A=a, scale_a=sa, B=b, scale_b=sb, D=d)
    dg.gemm_fp8(**good)
    for bad in (dict(A=a[:, :255]), dict(A=a.view(torch.uint8)), dict(scale_a=sa[:, :1]),
                dict(scale_b=sb[:1]), dict(D=d.int()), dict(D=d.t()), dict(D=d.cpu()),
                dict(scale_a=sa.double()), dict(bias=d[0].float(), epilogue="bias"),
                dict(bias=d[0, :5], epilogue="bias")):
        with pytest.raises((TypeError, ValueError)):
            dg.gemm_fp8(**{**good, **bad})
    for bad in (dict(epilogue="bias"), dict(epilogue=9), dict(alpha=float("inf"))):
        with pytest.raises(dg.DgError):
            dg.gemm_fp8(**{**good, **bad})
    x = torch.zeros(20, 256, dtype=torch.float16, device="cuda")
    for kw in (dict(form="columns"), dict(block_rows=64), dict(out=(a, sa, a)),
               dict(out=(a[:5], sa))):
        with pytest.raises((TypeError, ValueError)):
            dg.quantize_fp8(x, **kw)
    with pytest.raises(TypeError):
        dg.quantize_fp8(x.float())
    with pytest.raises(dg.DgError):
        dg.quantize_fp8(x[:, 1:200])  # not 16-byte aligned
    offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    w = torch.zeros(2, 256, 256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    ws = torch.zeros(2, 2, 2, device="cuda")
    dg.gemm_fp8_grouped(a, sa, w, ws, offsets, d)
    for args in ((a, sa, w, ws, offsets[:2], d), (a, sa, w, ws, offsets.long(), d),
                 (a, sa, w[:, :100], ws, offsets, d), (a, sa, w, ws[:1], offsets, d)):
        with pytest.raises((TypeError, ValueError)):
            dg.gemm_fp8_grouped(*args)
