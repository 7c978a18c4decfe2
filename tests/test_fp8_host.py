"""Argument checks of the FP8 and expert-routing entry points that need no GPU:
each refusal names what is wrong before any device is looked for."""

import pytest


@pytest.fixture(scope="module")
def dg():
    import __graft_entry__
    __graft_entry__.build()
    import precision_matmul_dg_gb300 as m
    return m


P = 0x10000  # an aligned address that no check looks behind


def refused(dg, status, word):
    assert dg.STATUS[status] in ("DG_ERR_INVALID_ARG", "DG_ERR_UNSUPPORTED"), (status, dg.last_error())
    assert word in dg.last_error(), dg.last_error()


def test_quantize(dg):
    def call(**kw):
        a = dict(rows=4, K=256, t=0, X=P, ldx=256, br=1, q=P, ldq=256, s=P, lds=2, qt=None, ldqt=0,
                 st=None, ldst=0)
        a.update(kw)
        return dg.lib().dg_quantize_fp8(*a.values(), None)
    for kw, word in ((dict(rows=-1), "negative"), (dict(K=1 << 31), "2^30"), (dict(t=1), "F16 or BF16"),
                     (dict(br=2), "block_rows"), (dict(X=None), "X is null"),
                     (dict(X=P + 2), "aligned"), (dict(ldx=255), "pitch"), (dict(ldx=260), "multiple of 8"),
                     (dict(q=None), "no output"), (dict(q=P + 8), "aligned"), (dict(ldq=250), "pitch"),
                     (dict(ldq=264), "multiple of 16"), (dict(s=None), "null"), (dict(lds=1), "need 2"),
                     (dict(s=P + 2), "4-byte"), (dict(qt=P, st=P, ldqt=3, ldst=1), "transposed")):
        refused(dg, call(**kw), word)
    for kw in (dict(rows=0), dict(K=0)):
        assert call(**kw) == 0


def test_gemm(dg):
    def call(**kw):
        a = dict(M=4, N=300, K=256, A=P, lda=256, sa=P, lds_a=2, B=P, ldb=256, sb=P, lds_b=2, br=128,
                 D=P, t=0, ldd=300, bias=None, alpha=1.0, beta=0.0, epi=0)
        a.update(kw)
        return dg.lib().dg_gemm_fp8(*a.values(), None)
    for kw, word in ((dict(M=-1), "negative"), (dict(br=3), "block_rows_b"), (dict(D=None), "D is null"),
                     (dict(t=1), "F16, BF16 or F32"), (dict(ldd=299), "ldd"), (dict(epi=7), "epilogue"),
                     (dict(epi=1), "null bias"), (dict(epi=1, bias=P + 1), "bias"),
                     (dict(beta=float("nan")), "finite"), (dict(A=P + 1), "A is not"),
                     (dict(B=None), "B or its"), (dict(ldb=257), "B: row pitch"),
                     (dict(lds_a=1), "A: 1 scales")):
        refused(dg, call(**kw), word)
    for kw in (dict(M=0), dict(N=0)):
        assert call(**kw) == 0


def test_grouped(dg):
    def call(**kw):
        a = dict(count=2, rows=40, N=300, K=256, A=P, lda=256, sa=P, lds_a=2, B=P, ldb=256,
                 stride_b=300 * 256, sb=P, lds_b=2, stride_sb=6, off=P, D=P, t=0, ldd=300, bias=None,
                 stride_bias=0, alpha=1.0, beta=0.0, epi=0)
        a.update(kw)
        return dg.lib().dg_gemm_fp8_grouped(*a.values(), None)
    for kw, word in ((dict(count=-1), "negative"), (dict(count=1025), "experts"),
                     (dict(off=None), "offsets"), (dict(stride_b=300 * 256 + 16), "stride_b"),
                     (dict(stride_b=299 * 256), "stride_b"), (dict(stride_sb=5), "stride_sb"),
                     (dict(N=1 << 30, stride_b=256 << 30, ldd=1 << 30, count=4, stride_sb=1 << 40),
                      "2^31")):
        refused(dg, call(**kw), word)
    for kw in (dict(count=0), dict(rows=0), dict(N=0)):
        assert call(**kw) == 0

    def grad(**kw):
        a = dict(count=2, M=8, N=16, rows=256, A=P, lda=256, sa=P, lds_a=2, B=P, ldb=256, sb=P,
                 lds_b=2, off=P, D=P, t=5, ldd=16, stride_d=128, alpha=1.0, beta=0.0)
        a.update(kw)
        return dg.lib().dg_gemm_fp8_grouped_wgrad(*a.values(), None)
    for kw, word in ((dict(count=1025), "experts"), (dict(stride_d=100), "stride_d"),
                     (dict(off=None), "offsets"), (dict(lda=200), "A: row pitch"),
                     (dict(t=2), "F16, BF16 or F32")):
        refused(dg, grad(**kw), word)
    assert grad(count=0) == 0


def test_routing(dg):
    L = dg.lib()
    assert L.dg_moe_rows(10, 2, 4, 1) == 20
    assert L.dg_moe_rows(10, 2, 4, 8) == 48  # 20 + 4 * 7
    assert L.dg_moe_rows(1, 2, 64, 128) == 256  # two experts at most have a row
    assert L.dg_moe_rows(0, 2, 64, 128) == 0
    assert L.dg_moe_rows(-1, 2, 64, 1) == -1 and L.dg_moe_rows(1, 0, 64, 1) == -1
    for args, word in (((-1, 2, 4, P, 1, 40, P, P, P), "tokens"), ((4, 2, 0, P, 1, 40, P, P, P), "count"),
                       ((4, 2, 1025, P, 1, 40, P, P, P), "experts"),
                       ((4, 2, 4, P, 3, 40, P, P, P), "align"), ((4, 2, 4, P, 1, 7, P, P, P), "7 rows"),
                       ((4, 2, 4, None, 1, 8, P, P, P), "null"),
                       ((4, 2, 4, P + 1, 1, 8, P, P, P), "4-byte")):
        refused(dg, L.dg_moe_sort(*args, None), word)
    for args, word in (((4, 2, 64, 1, P, 64, 8, P, P, 64), "F16 or BF16"),
                       ((4, 0, 64, 0, P, 64, 8, P, P, 64), "top_k"),
                       ((4, 2, 64, 0, P, 60, 8, P, P, 64), "X: row pitch"),
                       ((4, 2, 64, 0, P, 64, 8, None, P, 64), "row_slot"),
                       ((4, 2, 64, 0, P, 64, 8, P, P + 2, 64), "D is not")):
        refused(dg, L.dg_moe_dispatch(*args, None), word)
    refused(dg, L.dg_moe_dispatch_fp8(4, 2, 64, 0, P, 64, 8, P, P, 60, P, 1, None), "codes")
    refused(dg, L.dg_moe_combine(4, 2, 64, 0, P, 64, 8, None, P, P, 64, None), "slot_row")
    refused(dg, L.dg_moe_combine(4, 2, 64, 0, P, 64, 8, P, P + 2, P, 64, None), "weights")
    refused(dg, L.dg_moe_combine_backward(4, 2, 64, 0, P, 64, None, 64, 8, P, P, P, P, 64, P, None), "Y")
    assert L.dg_moe_dispatch(4, 2, 64, 0, P, 64, 0, P, P, 64, None) == 0
    assert L.dg_moe_combine(0, 2, 64, 0, P, 64, 8, P, P, P, 64, None) == 0
