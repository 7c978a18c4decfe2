"""64-bit references of the FP8 (E4M3, block scales) and expert-routing
operators, written from their definitions in include/dg.h with numpy only.

E4M3: value = (-1)^s * 2^(max(e, 1) - 7) * (m / 8 + [e > 0]); 0x7F and 0xFF
are NaN.  Blocks: 1 x 128 or 128 x 128 along K, one FP32 scale each.
"""

import numpy as np

BLOCK = 128
TOP = np.float32(448.0)
FLOOR = np.float32(448.0 * 2.0 ** -126)


def e4m3_values():
    """The 256 codes' values (float64; NaN for 0x7F and 0xFF)."""
    code = np.arange(256)
    e, m = (code >> 3) & 15, code & 7
    v = np.exp2(np.maximum(e, 1) - 7.0) * (m / 8.0 + (e > 0))
    v = np.where(code >= 128, -v, v)
    v[[0x7F, 0xFF]] = np.nan
    return v


VALUES = e4m3_values()


def e4m3_codes(x):
    """Nearest codes of finite x, ties to the even code, magnitudes above 448
    saturated, by search over the table (the sign of zero is kept)."""
    x = np.asarray(x, dtype=np.float64)
    grid = VALUES[:0x7F]
    mag = np.minimum(np.abs(x), grid[-1])
    hi = np.clip(np.searchsorted(grid, mag), 1, 0x7E)
    lo = hi - 1
    down, up = mag - grid[lo], grid[hi] - mag
    code = np.where(down < up, lo, np.where(up < down, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | (np.signbit(x) * 128)).astype(np.uint8)


def quantize(x, block_rows=1):
    """(codes uint8, scales float32) of x [rows, K], blocks along K; the two
    quotients and the product rounded to float32 as the definition says."""
    x = np.asarray(x, dtype=np.float32)
    rows, K = x.shape
    codes = np.zeros((rows, K), np.uint8)
    scales = np.zeros((-(-rows // block_rows), -(-K // BLOCK)), np.float32)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = np.s_[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]
            b = x[at]
            if not np.isfinite(b).all():
                scales[i, j] = np.nan
                continue
            amax = max(np.float32(np.abs(b).max()), FLOOR)
            scales[i, j] = amax / TOP
            codes[at] = e4m3_codes(b * (TOP / amax))
    return codes, scales


def values(codes, scales, block_rows=1):
    """What the codes stand for, float64."""
    s = np.repeat(np.asarray(scales, np.float64), BLOCK, 1)[:, :codes.shape[1]]
    return VALUES[codes] * np.repeat(s, block_rows, 0)[:codes.shape[0]]


def gelu(t):
    from .gemm_ref import gelu_erf
    return gelu_erf(t)


def product(a, b, alpha=1.0, beta=0.0, d=None, bias=None, use_gelu=False):
    """epilogue(alpha * a.b^T + beta * d) of values a [M, K], b [N, K], and the
    error bound of an FP32 computation before its last rounding.

    The products of two E4M3 values are exact in FP32.  A block's 128 are added
    in FP32 (truncation allowed: 2^-23 each), then scaled (two roundings) and
    added block by block: at most (128 + 3 + blocks) * 2^-23 of the sum of
    magnitudes.  alpha, beta and bias add a rounding each; GELU's slope is at
    most 1.13 and its evaluation good to 2e-7 of |t|."""
    t = a @ b.T
    mags = np.abs(a) @ np.abs(b).T
    blocks = -(-a.shape[1] // BLOCK)
    u = 2.0 ** -23
    err = abs(alpha) * mags * (128 + 4 + blocks) * u
    t = alpha * t
    if beta != 0.0:
        t = t + beta * d
        err = err + (np.abs(t) + np.abs(beta * d)) * u
    if bias is not None:
        t = t + bias
        err = err + (np.abs(t) + np.abs(bias)) * u
    if use_gelu:
        err = 1.13 * err + 2e-7 * np.abs(t)
        t = gelu(t)
    return t, err


HALF_ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -149}


def rounded_bound(ref, err, dtype):
    """err and one rounding to dtype (half an ulp of the result; bfloat16 has 8
    significant bits)."""
    return err + (np.abs(ref) + err) * HALF_ULP[dtype] + TINY[dtype]


def sort_by_expert(ids, count, align=1, rows=None):
    """(offsets, row_slot, slot_row) by a loop over experts and slots."""
    flat = np.asarray(ids).reshape(-1)
    offsets, row_slot = [0], []
    for e in range(count):
        mine = [s for s, v in enumerate(flat) if v == e]
        row_slot += mine + [-1] * (-len(mine) % align)
        offsets.append(len(row_slot))
    if rows is not None:
        row_slot += [-1] * (rows - len(row_slot))
    slot_row = np.full(flat.shape, -1, np.int32)
    for r, s in enumerate(row_slot):
        if s >= 0:
            slot_row[s] = r
    return (np.array(offsets, np.int32), np.array(row_slot, np.int32),
            slot_row.reshape(np.shape(ids)))


def dispatch(x, row_slot, top_k):
    out = np.zeros((len(row_slot), x.shape[1]))
    for r, s in enumerate(row_slot):
        if s >= 0:
            out[r] = x[s // top_k]
    return out


def combine(y, slot_row, weights=None):
    """The sum and the sum of magnitudes (for error bounds)."""
    tokens, top_k = slot_row.shape
    out, mags = np.zeros((tokens, y.shape[1])), np.zeros((tokens, y.shape[1]))
    for t in range(tokens):
        for j in range(top_k):
            if slot_row[t, j] >= 0:
                v = (1.0 if weights is None else float(weights[t, j])) * y[slot_row[t, j]]
                out[t] += v
                mags[t] += np.abs(v)
    return out, mags


def combine_backward(dd, y, slot_row, rows, weights=None):
    tokens, top_k = slot_row.shape
    dy, dw = np.zeros((rows, dd.shape[1])), np.zeros((tokens, top_k))
    for t in range(tokens):
        for j in range(top_k):
            r = slot_row[t, j]
            if r >= 0:
                dy[r] = (1.0 if weights is None else float(weights[t, j])) * dd[t]
                dw[t, j] = dd[t] @ y[r]
    return dy, dw
