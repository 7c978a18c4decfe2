"""Argument checks of the NVF4 operators and of the expert layer that need no
GPU: each refusal names what is wrong before any device is looked for."""

import ctypes

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
        a = dict(count=2, rows=4, K=250, t=0, X=P, ldx=256, stride_x=1024, given=None, q=P, ldq=128,
                 stride_q=512, s=P, r=P)
        a.update(kw)
        return dg.lib().dg_quantize_nvf4(*a.values(), None)
    for kw, word in ((dict(rows=-1), "negative"), (dict(K=1 << 31), "2^30"), (dict(t=5), "F16 or BF16"),
                     (dict(X=None), "X is null"), (dict(X=P + 2), "aligned"), (dict(ldx=248), "pitch"),
                     (dict(ldx=252), "multiple of 8"), (dict(stride_x=1016), "stride"),
                     (dict(stride_x=1028), "multiple of 8"), (dict(q=None), "null"),
                     (dict(q=P + 8), "aligned"), (dict(ldq=124), "pitch"), (dict(ldq=136), "multiple of 16"),
                     (dict(stride_q=500), "stride"), (dict(s=P + 4), "aligned"), (dict(s=None), "null"),
                     (dict(r=None), "null"), (dict(r=P + 2), "4-byte"), (dict(given=P + 2), "4-byte"),
                     (dict(count=1 << 30, rows=1 << 30, stride_x=1 << 40, stride_q=1 << 40), "2^40")):
        refused(dg, call(**kw), word)
    for kw in (dict(rows=0), dict(K=0), dict(count=0)):
        assert call(**kw) == 0


def test_dispatch(dg):
    def call(**kw):
        a = dict(tokens=4, top_k=2, width=250, t=1, X=P, ldx=256, rows=8, slot=P, q=P, ldq=128, s=P, r=P)
        a.update(kw)
        a["t"] = {1: dg.BF16, 0: dg.F16}.get(a["t"], a["t"])
        return dg.lib().dg_moe_dispatch_nvf4(*a.values(), None)
    for kw, word in ((dict(top_k=0), "top_k"), (dict(t=5), "F16 or BF16"), (dict(slot=None), "row_slot"),
                     (dict(ldx=249), "X: row pitch"), (dict(ldq=100), "codes"), (dict(r=None), "null")):
        refused(dg, call(**kw), word)
    assert call(rows=0) == 0


def test_dequantize(dg):
    def call(**kw):
        a = dict(count=2, rows=4, K=250, q=P, ldq=128, stride_q=512, s=P, r=P, D=P, t=5, ldd=251,
                 stride_d=1003)
        a.update(kw)
        return dg.lib().dg_dequantize_nvf4(*a.values(), None)
    for kw, word in ((dict(t=1), "F16, BF16 or F32"), (dict(ldd=249), "ldd"), (dict(D=None), "D is null"),
                     (dict(D=P + 2), "aligned to its type"), (dict(stride_d=1002), "overlap"),
                     (dict(stride_q=448), "stride"), (dict(ldq=120), "pitch")):
        refused(dg, call(**kw), word)
    assert call(rows=0) == 0


def test_gemm(dg):
    def call(**kw):
        a = dict(M=4, N=300, K=250, A=P, lda=128, sa=P, ra=P, B=P, ldb=128, sb=P, rb=P, D=P, t=0,
                 ldd=300, bias=None, alpha=1.0, beta=0.0, epi=0)
        a.update(kw)
        return dg.lib().dg_gemm_nvf4(*a.values(), None)
    for kw, word in ((dict(M=-1), "negative"), (dict(K=0), "at least 1"), (dict(D=None), "D is null"),
                     (dict(t=1), "F16, BF16 or F32"), (dict(ldd=299), "ldd"), (dict(epi=7), "epilogue"),
                     (dict(epi=1), "null bias"), (dict(epi=1, bias=P + 1), "bias"),
                     (dict(alpha=float("inf")), "finite"), (dict(A=P + 1), "A or its"),
                     (dict(B=None), "B or its"), (dict(ldb=124), "B: row pitch"), (dict(rb=P + 1), "B: row"),
                     (dict(M=1 << 30, K=1 << 30, lda=1 << 29, ldb=1 << 29), "2^31")):
        refused(dg, call(**kw), word)
    for kw in (dict(M=0), dict(N=0)):
        assert call(**kw) == 0


def test_grouped(dg):
    def call(**kw):
        a = dict(count=2, rows=256, N=300, K=250, A=P, lda=128, sa=P, ra=P, B=P, ldb=128,
                 stride_b=300 * 128, sb=P, rb=P, off=P, D=P, t=0, ldd=300, bias=None, stride_bias=0,
                 alpha=1.0, beta=0.0, epi=0)
        a.update(kw)
        return dg.lib().dg_gemm_nvf4_grouped(*a.values(), None)
    for kw, word in ((dict(count=-1), "negative"), (dict(count=1025), "experts"), (dict(K=0), "at least 1"),
                     (dict(off=None), "offsets"), (dict(off=P + 2), "offsets"),
                     (dict(stride_b=300 * 128 + 16), "stride_b"), (dict(stride_b=299 * 128), "stride_b"),
                     (dict(N=1 << 30, ldd=1 << 30, count=4, stride_b=128 << 30), "2^31"),
                     (dict(epi=1, bias=P, stride_bias=-1), "stride_bias")):
        refused(dg, call(**kw), word)
    for kw in (dict(count=0), dict(rows=0), dict(N=0)):
        assert call(**kw) == 0


def weights(dg, **kw):
    a = dict(codes=P, ld=256, stride=512 * 256, scales=P, lds=2, stride_s=8, row_scales=P, bias=None,
             stride_bias=0)
    a.update(kw)
    return dg.MoeWeights(*a.values())


def test_layer(dg):
    def call(up=None, down=None, **kw):
        a = dict(tokens=4, top_k=2, count=8, width=256, hidden=256, out=256, t=0, X=P, ldx=256, ids=P,
                 w=P, fmt=0, up=weights(dg) if up is None else up,
                 down=weights(dg) if down is None else down, act=0, D=P, ldd=256,
                 scratch=P, bytes=1 << 20)
        a.update(kw)
        return dg.lib().dg_moe_layer(*a.values(), None)
    for kw, word in ((dict(tokens=-1), "tokens"), (dict(top_k=0), "top_k"), (dict(tokens=257), "512"),
                     (dict(count=0), "count"), (dict(count=1025), "experts"), (dict(width=0), "at least 1"),
                     (dict(hidden=0), "at least 1"), (dict(out=1 << 25), "2^24"),
                     (dict(t=5), "F16 or BF16"), (dict(fmt=2), "format"), (dict(act=2), "activation"),
                     (dict(X=P + 2), "aligned"), (dict(ldx=250), "X: row pitch"), (dict(ldd=252), "D: row"),
                     (dict(ids=None), "ids"), (dict(w=P + 1), "weights"), (dict(scratch=None), "scratch"),
                     (dict(scratch=P + 8), "scratch"), (dict(bytes=100), "scratch, need"),
                     (dict(tokens=32, width=4096, ldx=4096, up=weights(dg, ld=4096, stride=1 << 21, lds=32,
                                                                       stride_s=64)), "shared memory"),
                     (dict(fmt=1, act=1, hidden=200), "multiple of 128"),
                     (dict(up=weights(dg, codes=None)), "up or its"),
                     (dict(up=weights(dg, ld=248)), "up: row pitch"),
                     (dict(up=weights(dg, lds=1)), "up: 1 scales"),
                     (dict(down=weights(dg, stride=255 * 256)), "down: stride"),
                     (dict(down=weights(dg, stride_s=3)), "down: stride_s"),
                     (dict(up=weights(dg, codes=P + 4)), "aligned"),
                     (dict(fmt=1, up=weights(dg, row_scales=None)), "up or its"),
                     (dict(fmt=1, up=weights(dg, scales=P + 8)), "aligned"),
                     (dict(up=weights(dg, bias=P + 1)), "bias"),
                     (dict(up=weights(dg, bias=P, stride_bias=-1)), "stride_bias"),
                     (dict(act=1, up=weights(dg, stride=256 * 256)), "up: stride")):
        refused(dg, call(**kw), word)
    none = ctypes.POINTER(dg.MoeWeights)()
    refused(dg, call(up=none), "up is null")
    for kw in (dict(tokens=0), dict(out=0)):
        assert call(**kw) == 0
    L = dg.lib()
    assert L.dg_moe_layer_scratch(4, 2, 256, 256) > 8 * 256 * 2
    for sizes in ((-1, 2, 256, 256), (4, 0, 256, 256), (513, 1, 256, 256), (4, 2, -1, 256)):
        assert L.dg_moe_layer_scratch(*sizes) == -1


def test_binding_refuses(dg):
    """What the binding turns away before it calls the library: host tensors, wrong types,
    shapes and strides."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.float16)
    buf = dg.nvf4_buffers(4, 64, device="cpu")
    assert [tuple(t.shape) for t in buf] == [(4, 32), (1, 1, 32, 16), (4,)]
    assert buf[0].stride() == (32, 1) and dg.nvf4_buffers(3, 5, 33, device="cpu")[0].shape == (3, 5, 17)
    d = torch.zeros(4, 4, dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU"):
        dg.quantize_nvf4(x, out=buf)
    with pytest.raises(TypeError, match="float16"):
        dg.quantize_nvf4(x.double(), out=buf)
    with pytest.raises(ValueError, match="GPU"):
        dg.gemm_nvf4(*buf, *buf, d)
    with pytest.raises(TypeError, match="uint8"):
        dg.gemm_nvf4(buf[0].to(torch.int8), *buf[1:], *buf, d)
    with pytest.raises(ValueError):
        dg.dequantize_nvf4(buf[0][:, :30], buf[1], buf[2], x)
    with pytest.raises((ValueError, TypeError)):
        dg.moe_layer(x, torch.zeros(4, 2, dtype=torch.int32), None, buf, buf, x)
