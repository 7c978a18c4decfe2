"""64-bit references of the 4-bit operators with E4M3 block scales and of the
expert layer for a few tokens, written from their definitions in include/dg.h
with numpy only.

A value is e2m1(code) * e4m3(scale) * row_scale: one E4M3 scale per 16 values
along K, one FP32 scale per row.  Codes are packed two to a byte; scales lie in
tiles of 128 rows x 4 blocks.
"""

import numpy as np

from . import fp8_ref

GROUP = 16
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])  # magnitudes of codes 0 .. 7
NAN = 0x7F


def e2m1_codes(x):
    """Nearest codes of x, ties to the even code, saturated at 6, signs kept."""
    x = np.asarray(x, np.float64)
    mag = np.minimum(np.abs(x), 6.0)
    hi = np.clip(np.searchsorted(GRID, mag), 1, 7)
    lo = hi - 1
    down, up = mag - GRID[lo], GRID[hi] - mag
    code = np.where(down < up, lo, np.where(up < down, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | (np.signbit(x) * 8)).astype(np.uint8)


def row_scale(amax):
    """The smallest power of two r >= 2^-100 with 2688 r >= amax."""
    e = -100
    while 2688.0 * 2.0 ** e < amax:
        e += 1
    return np.float32(2.0 ** e)


def quantize(x, given=None):
    """(codes [rows, K], one to a byte, scale codes [rows, groups], row scales) of
    x [rows, K]; quotients and products rounded to float32 as the definition says."""
    x = np.asarray(x, np.float32)
    rows, K = x.shape
    groups = -(-K // GROUP)
    full = np.zeros((rows, groups * GROUP), np.float32)
    full[:, :K] = x
    v = full.reshape(rows, groups, GROUP)
    fine = np.isfinite(v).all(2)
    amax = np.abs(np.where(fine[..., None], v, 0)).max(2)
    if given is None:
        r = np.array([row_scale(float(a)) for a in amax.max(1)], np.float32)
        ok = np.ones(rows, bool)
    else:
        r = np.asarray(given, np.float32)
        ok = (r >= 2.0 ** -100) & (r <= 2.0 ** 100)
    safe = np.where(ok, r, np.float32(1))[:, None]
    with np.errstate(over="ignore", invalid="ignore"):
        scales = np.maximum(fp8_ref.e4m3_codes(amax / (np.float32(6.0) * safe)), 1)
        u = fp8_ref.VALUES[scales].astype(np.float32) * safe
        codes = e2m1_codes(v / u[..., None])
    good = fine & ok[:, None]
    codes = np.where(good[..., None], codes, 0).astype(np.uint8)
    return (codes.reshape(rows, -1)[:, :K], np.where(good, scales, NAN).astype(np.uint8), r)


def pack(codes):
    """Two codes to a byte, the even one in the low nibble."""
    rows, K = codes.shape
    full = np.zeros((rows, K + K % 2), np.uint8)
    full[:, :K] = codes
    return full[:, 0::2] | (full[:, 1::2] << 4)


def unpack(packed, K):
    codes = np.zeros(packed.shape[:-1] + (2 * packed.shape[-1],), np.uint8)
    codes[..., 0::2] = packed & 15
    codes[..., 1::2] = packed >> 4
    return codes[..., :K]


def tiles(scales):
    """Scale codes [rows, groups] in tiles, group by group."""
    rows, groups = scales.shape
    out = np.zeros((-(-rows // 128), -(-groups // 4), 32, 16), np.uint8)
    r = np.arange(rows)
    for g in range(groups):
        out[r // 128, g // 4, r % 32, 4 * (r % 128 // 32) + g % 4] = scales[:, g]
    return out


def values(codes, scales, rows_scale):
    """What codes [rows, K] with scale codes [rows, groups] stand for, float64."""
    mag = GRID[codes & 7]
    v = np.where(codes > 7, -mag, mag)
    s = np.repeat(fp8_ref.VALUES[scales], GROUP, 1)[:, :codes.shape[1]]
    return v * s * np.asarray(rows_scale, np.float64)[:, None]


def product(a, b, alpha=1.0, beta=0.0, d=None, bias=None, use_gelu=False):
    """epilogue(alpha * a.b^T + beta * d) of values a [M, K], b [N, K], and the
    error bound of an FP32 computation before its last rounding.

    A product of two scaled values is exact in FP32 (at most 4 + 8 significant
    bits).  The K of them are added in FP32 (truncation allowed: 2^-23 each) and
    scaled by both rows' scales (two roundings, alpha's with the row's a third).
    beta and bias add a rounding each; GELU's slope is at most 1.13 and its
    evaluation good to 2e-7 of |t|."""
    t = alpha * (a @ b.T)
    mags = abs(alpha) * (np.abs(a) @ np.abs(b).T)
    u = 2.0 ** -23
    err = mags * (a.shape[1] + 4) * u
    if beta != 0.0:
        t = t + beta * d
        err = err + (np.abs(t) + np.abs(beta * d)) * u
    if bias is not None:
        t = t + bias
        err = err + (np.abs(t) + np.abs(bias)) * u
    if use_gelu:
        err = 1.13 * err + 2e-7 * np.abs(t)
        t = fp8_ref.gelu(t)
    return t, err


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def chain(K):
    """Roundings (or truncations) to 24 bits that a term of the layer's sums of K products
    passes, and those that the sum's other terms pass beside it, at most.

    The products are taken by MMAs of 16 with an accumulator: an exact product of two
    FP16 values, then 16 of them and the accumulator aligned to the largest, added and
    normalised, 18 truncations.  A term passes up to eight of them (256 values of K in
    4 bits, which two accumulators share; 2 for each 32 values, whose halves lie in both),
    then FP32 additions: of the accumulators, times scales, into the sum of the blocks that
    a warp meets, which are every second at least (up to 5 for each 512 values: in 8
    bits, one for each of the four powers of h in a block and one for the block), up to
    eight warps' sums, h's two values' sums, and the row's scale.  Additions of zeros, past
    K, are exact."""
    return 18 * min(8, 2 * -(-K // 32)) + 5 * -(-K // 512) + 10


def layer(x, ids, weights, up, down, gated=False, bias_up=None, bias_down=None):
    """(y, bound) of the expert layer on values: x [tokens, width], up [count,
    hidden or 2 hidden, width], down [count, out, hidden]; the bound is of an
    FP32 computation with x and h held as include/dg.h says, before the last
    rounding.

    A product errs by chain(K) roundings of 2^-23 of the sum of magnitudes, a value of x
    by 2^-39 of its row's largest, one of h (two FP16 values, the second what the first
    leaves) by 2^-22 of itself and 2^-39 of the largest of 32 around it.  GELU's and
    SiLU's slopes are at most 1.13, and they are evaluated to 2e-6."""
    tokens, top_k = ids.shape
    count, out = down.shape[0], down.shape[1]
    u = 2.0 ** -23
    y, bound = np.zeros((tokens, out)), np.zeros((tokens, out))

    def product(W, v, verr, bias):
        t = W @ v
        mags = np.abs(W) @ np.abs(v)
        err = mags * chain(len(v)) * u + np.abs(W) @ verr
        if bias is not None:
            t = t + bias
            err = err + (np.abs(t) + np.abs(bias)) * u
        return t, err
    for t in range(tokens):
        for j in range(top_k):
            e = ids[t, j]
            if not 0 <= e < count:
                continue
            h, err = product(up[e], x[t], np.full(x.shape[1], np.abs(x[t]).max() * 2.0 ** -39),
                             None if bias_up is None else bias_up[e])
            if gated:
                n = len(h) // 2
                g, v = h[:n], h[n:]
                eg, ev = err[:n], err[n:]
                s = silu(g)
                es = 1.13 * eg + 2e-6 * np.abs(s)
                h = s * v
                err = es * np.abs(v) + (np.abs(s) + es) * ev + np.abs(h) * u
            else:
                err = 1.13 * err + 2e-6 * np.abs(h)
                h = fp8_ref.gelu(h)
            pad = np.zeros(-len(h) % 32)
            around = np.repeat(np.concatenate([np.abs(h) + err, pad]).reshape(-1, 32).max(1), 32)
            err = err + 2.0 ** -22 * (np.abs(h) + err) + 2.0 ** -39 * around[:len(h)]
            v, ev = product(down[e], h, err, None if bias_down is None else bias_down[e])
            w = 1.0 if weights is None else float(weights[t, j])
            y[t] += w * v
            bound[t] += abs(w) * (ev + np.abs(v) * (top_k + 1) * u)
    return y, bound
