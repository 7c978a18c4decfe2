"""Expert routing: the sort exactly, rows there exactly (or quantized bit for
bit), rows back and their gradient within FP32 sums and one rounding."""

import numpy as np
import pytest
import torch

from oracle import fp8_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def dg():
    import precision_matmul_dg_gb300 as m
    m.lib()
    return m


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def some_ids(tokens, top_k, count, seed, bad=0.0):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, count, (tokens, top_k)).astype(np.int32)
    ids[rng.random(ids.shape) < bad] = -1
    ids[rng.random(ids.shape) < bad / 2] = count + 3
    return ids


@pytest.mark.parametrize("align", [1, 2, 128])
@pytest.mark.parametrize("tokens,top_k,count,bad", [
    (0, 2, 4, 0.0), (1, 1, 1, 0.0), (8, 8, 64, 0.0), (100, 2, 3, 0.3), (33, 1, 1000, 0.1),
    (5000, 3, 16, 0.05), (40, 2, 1024, 1.0), (20000, 8, 128, 0.02)])
def test_sort(dg, tokens, top_k, count, bad, align):
    ids = some_ids(tokens, top_k, count, tokens + count, bad)
    got = dg.moe_sort(gpu(ids), count, align=align)
    dg.check_status()
    want = ref.sort_by_expert(ids, count, align, dg.moe_rows(tokens, top_k, count, align))
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)


def test_sort_into_a_larger_buffer(dg):
    ids = some_ids(50, 2, 8, 3, 0.2)
    out = (torch.full((9,), 5, dtype=torch.int32, device="cuda"),
           torch.full((5000,), 5, dtype=torch.int32, device="cuda"),
           torch.full((50, 2), 5, dtype=torch.int32, device="cuda"))
    dg.moe_sort(gpu(ids), 8, out=out)
    for g, w in zip(out, ref.sort_by_expert(ids, 8, 1, 5000)):
        assert np.array_equal(g.cpu().numpy(), w)


def rows16(rows, width, seed, dtype, pad=8):
    ld = (width + 7) // 8 * 8 + pad
    x = torch.randn(rows, ld, generator=torch.Generator().manual_seed(seed)).to(TYPES[dtype])
    return x.cuda()[:, :width], x[:, :width].double().numpy()


CASES = [(1, 1, 1, 8), (8, 8, 64, 2048), (37, 3, 5, 100), (300, 2, 16, 257), (20, 11, 4, 1000),
         (64, 16, 20, 33), (5, 2, 3, 1)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("align", [1, 128])
@pytest.mark.parametrize("tokens,top_k,count,width", CASES)
def test_there_and_back(dg, tokens, top_k, count, width, align, dtype):
    ids = some_ids(tokens, top_k, count, width, 0.15)
    offsets, row_slot, slot_row = dg.moe_sort(gpu(ids), count, align=align)
    rows = row_slot.shape[0]
    rs, sr = row_slot.cpu().numpy(), slot_row.cpu().numpy()
    x, x64 = rows16(tokens, width, 1, dtype)
    t = TYPES[dtype]
    # there
    room = torch.full((rows, (width + 7) // 8 * 8 + 8), 3.0, dtype=t, device="cuda")
    dg.moe_dispatch(x, row_slot, top_k, room[:, :width])
    want = ref.dispatch(x64, rs, top_k)
    assert np.array_equal(room[:, :width].double().cpu().numpy(), want)
    assert (room[:, width:] == 3.0).all()
    # there, quantized
    codes = torch.zeros(rows, (width + 15) // 16 * 16, dtype=torch.uint8,
                        device="cuda").view(torch.float8_e4m3fn)[:, :width]
    scales = torch.zeros(rows, -(-width // 128), device="cuda")
    dg.moe_dispatch_fp8(x, row_slot, top_k, codes, scales)
    qc, qs = ref.quantize(want)
    got = codes.cpu().contiguous().view(torch.uint8).numpy()
    assert np.array_equal(ref.VALUES[got], ref.VALUES[qc])
    assert np.array_equal(scales.cpu().numpy(), qs)
    # back
    y, y64 = rows16(rows, width, 2, dtype)
    w = torch.randn(tokens, top_k, generator=torch.Generator().manual_seed(3)).cuda()
    for weights in (w, None):
        room = torch.full((tokens, (width + 7) // 8 * 8), 3.0, dtype=t, device="cuda")
        dg.moe_combine(y, slot_row, room[:, :width], weights=weights)
        out, mags = ref.combine(y64, sr, None if weights is None else w.cpu().numpy())
        err = np.abs(room[:, :width].double().cpu().numpy() - out)
        assert (err <= ref.rounded_bound(out, mags * (top_k + 1) * 2.0 ** -24, dtype)).all()
        assert (room[:, width:] == 3.0).all()
    # and its gradient
    dd, dd64 = rows16(tokens, width, 4, dtype)
    for weights in (w, None):
        dy = torch.full((rows, (width + 7) // 8 * 8), 3.0, dtype=t, device="cuda")
        dw = torch.full((tokens, top_k), 3.0, device="cuda")
        dg.moe_combine_backward(dd, y, slot_row, row_slot, weights, dy[:, :width], dw)
        dg.check_status()
        w64 = None if weights is None else w.cpu().numpy()
        rdy, rdw = ref.combine_backward(dd64, y64, sr, rows, w64)
        err = np.abs(dy[:, :width].double().cpu().numpy() - rdy)
        # the product rounded to FP32, then to the type
        assert (err <= ref.rounded_bound(rdy, np.abs(rdy) * 2.0 ** -24, dtype)).all()
        _, mags = ref.combine_backward(np.abs(dd64), np.abs(y64), sr, rows, w64)
        assert (np.abs(dw.double().cpu().numpy() - rdw) <= mags * (width + 2) * 2.0 ** -24).all()
        only = torch.full_like(dy, 3.0)
        dg.moe_combine_backward(dd, None, slot_row, row_slot, weights, only[:, :width])
        assert torch.equal(only, dy)


def test_no_tokens(dg):
    e = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    offsets, row_slot, slot_row = dg.moe_sort(e, 4, align=128)
    assert (offsets == 0).all() and row_slot.shape == (0,)
    x = torch.zeros(0, 64, dtype=torch.float16, device="cuda")
    assert dg.moe_dispatch(x, row_slot, 2, torch.zeros_like(x)).shape == (0, 64)
    assert dg.moe_combine(x, slot_row, torch.zeros_like(x)).shape == (0, 64)


def test_long_rows_pass_32_bits(dg):
    # 70000 rows of 40000 values: element offsets past 2^31
    rows, width = 70000, 40000
    y = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    y[rows - 1] = 2.0
    slot_row = torch.tensor([[rows - 1, 0]], dtype=torch.int32, device="cuda")
    d = torch.zeros(1, width, dtype=torch.bfloat16, device="cuda")
    dg.moe_combine(y, slot_row, d)
    assert (d == 2.0).all()
    row_slot = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    row_slot[rows - 1] = 0
    dg.moe_dispatch(d, row_slot, 2, y)
    assert (y[rows - 1] == 2.0).all() and (y[:5] == 0.0).all()
    del y


def test_refusals(dg):
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    for args, kw in (((ids.long(), 4), {}), ((ids.t(), 4), {}), ((ids.cpu(), 4), {}),
                     ((ids, 4), dict(align=0))):
        with pytest.raises((TypeError, ValueError, dg.DgError)):
            dg.moe_sort(*args, **kw)
    offsets, row_slot, slot_row = dg.moe_sort(ids, 4)
    for kw in (dict(align=3), dict(align=2), dict(out=(offsets, row_slot[:5], slot_row))):
        with pytest.raises(dg.DgError):
            dg.moe_sort(ids, 4, **{**dict(out=(offsets, row_slot, slot_row)), **kw})
    with pytest.raises(dg.DgError):
        dg.moe_sort(ids, 2000)
    x = torch.zeros(4, 64, dtype=torch.float16, device="cuda")
    d = torch.zeros(8, 64, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        dg.moe_dispatch(x, row_slot, 2, d[:7])
    with pytest.raises(TypeError):
        dg.moe_dispatch(x, row_slot, 2, d.bfloat16())
    with pytest.raises(dg.DgError):
        dg.moe_dispatch(x[:, 1:33], row_slot, 2, d[:, :32])  # not 16-byte aligned
    with pytest.raises(ValueError):
        dg.moe_combine(d, slot_row, x[:3])
    with pytest.raises(ValueError):
        dg.moe_combine_backward(x, None, slot_row, row_slot, None, d,
                                torch.zeros(4, 2, device="cuda"))
