"""The expert layer of a few tokens on FP8 and NVF4 weights, against 64-bit
arithmetic within the bound that oracle.nvf4_ref.layer derives."""

import numpy as np
import pytest
import torch

from oracle import fp8_ref, nvf4_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
FORMATS = ["fp8", "nvf4"]


@pytest.fixture(scope="module")
def dg():
    import precision_matmul_dg_gb300 as m
    m.lib()
    return m


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def weights(fmt, count, n, k, rng, pad_rows=0):
    """A stack of weights on the GPU, NaN codes (or others) past the rows' ends and between
    matrices, and their values in 64 bits."""
    w = rng.normal(size=(count, n, k)) / k ** 0.5 * np.exp2(rng.integers(-1, 2, (count, n, 1)))
    if fmt == "fp8":
        parts = [fp8_ref.quantize(m, 128) for m in w]
        room = np.full((count, n + pad_rows, -(-k // 16) * 16 + 16), 0x7F, np.uint8)
        room[:, :n, :k] = np.stack([p[0] for p in parts])
        scales = np.stack([p[1] for p in parts])
        return ((gpu(room).view(torch.float8_e4m3fn)[:, :n, :k], gpu(scales)),
                np.stack([fp8_ref.values(p[0], p[1], 128) for p in parts]))
    codes, scales, rows = ref.quantize(w.reshape(count * n, k))
    parts = list(zip(codes.reshape(count, n, k), scales.reshape(count, n, -1)))
    room = np.full((count, n + pad_rows, -(-k // 32) * 16 + 16), 0x77, np.uint8)
    room[:, :n, :(k + 1) // 2] = ref.pack(codes).reshape(count, n, -1)
    rows = rows.reshape(count, n) * rng.uniform(0.6, 1.7, (count, n)).astype(np.float32)
    rows = rows.astype(np.float32)
    return ((gpu(room)[:, :n, :(k + 1) // 2],
             gpu(np.stack([ref.tiles(p[1]) for p in parts])).view(torch.float8_e4m3fn), gpu(rows)),
            np.stack([ref.values(p[0], p[1], r) for p, r in zip(parts, rows)]))


class Case:
    def __init__(self, fmt, tokens, top_k, count, width, hidden, out, dtype="bf16", gated=False,
                 bias=False, seed=0, ids=None, weighted=True, pad_rows=0):
        rng = np.random.default_rng(seed)
        t = TYPES[dtype]
        self.up, self.up64 = weights(fmt, count, hidden * (2 if gated else 1), width, rng, pad_rows)
        self.down, self.down64 = weights(fmt, count, out, hidden, rng, pad_rows)
        ld = -(-width // 8) * 8 + 8
        x = torch.from_numpy(rng.normal(size=(tokens, ld)) *
                             np.exp2(rng.integers(-3, 4, (tokens, 1)))).to(t)
        self.x, self.x64 = x.cuda()[:, :width], x[:, :width].double().numpy()
        if ids is None:
            ids = np.stack([rng.permutation(count)[:top_k] for _ in range(tokens)])
        self.ids64 = np.asarray(ids, np.int32)
        self.ids = gpu(self.ids64)
        w = rng.uniform(0.05, 1.0, self.ids64.shape).astype(np.float32)
        self.w64 = w if weighted else None
        self.w = gpu(w) if weighted else None
        self.bias = (None, None)
        self.bias64 = (None, None)
        if bias:
            b = [torch.from_numpy(rng.normal(size=(count, n))).to(t)
                 for n in (self.up64.shape[1], out)]
            self.bias, self.bias64 = [v.cuda() for v in b], [v.double().numpy() for v in b]
        self.room = torch.full((tokens, -(-out // 8) * 8 + 8), 7.0, dtype=t, device="cuda")
        self.d, self.gated, self.dtype = self.room[:, :out], gated, dtype

    def run(self, dg, **kw):
        return dg.moe_layer(self.x, self.ids, self.w, self.up, self.down, self.d,
                            activation="swiglu" if self.gated else "gelu", bias_up=self.bias[0],
                            bias_down=self.bias[1], **kw)

    def wanted(self):
        y, err = ref.layer(self.x64, self.ids64, self.w64, self.up64, self.down64, self.gated,
                           *self.bias64)
        return y, fp8_ref.rounded_bound(y, err, self.dtype)

    def check(self):
        y, bound = self.wanted()
        g = self.d.double().cpu().numpy()
        bad = ~(np.abs(g - y) <= bound)
        assert not bad.any(), "%d of %d outside the bound, first at %s: %r for %r, bound %r" % (
            bad.sum(), bad.size, np.argwhere(bad)[0], g[bad][0], y[bad][0], bound[bad][0])
        assert (self.room[:, self.d.shape[1]:] == 7.0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens,top_k,count,width,hidden,out,dtype,gated", [
    (1, 1, 1, 32, 32, 32, "f16", False),
    (1, 1, 1, 16, 128, 16, "bf16", True),
    (1, 2, 4, 256, 320, 256, "bf16", False),
    (2, 2, 4, 520, 256, 520, "f16", True),
    (3, 2, 5, 264, 100, 136, "f16", False),
    (5, 4, 6, 1000, 77, 1001, "bf16", False),
    (8, 2, 8, 512, 384, 512, "bf16", True),
    (16, 3, 4, 1024, 512, 264, "f16", True),
    (32, 4, 8, 136, 160, 72, "bf16", False),
    (4, 8, 16, 2048, 256, 2048, "bf16", True),
    (1, 8, 64, 2048, 128, 96, "f16", False),
    (2, 1, 3, 9, 8, 1, "bf16", False),
    (3, 2, 3, 1, 1, 33, "f16", False),
])
def test_layer(dg, fmt, tokens, top_k, count, width, hidden, out, dtype, gated):
    c = Case(fmt, tokens, top_k, count, width, hidden, out, dtype, gated, seed=tokens + width)
    c.run(dg)
    dg.check_status()
    c.check()
    first = c.d.clone()
    for _ in range(3):  # bit for bit
        c.run(dg)
        assert torch.equal(c.d, first)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("gated", [False, True])
def test_biases_strides_and_no_weights(dg, fmt, gated):
    c = Case(fmt, 6, 2, 5, 300 if fmt == "fp8" else 296, 128, 200, "bf16", gated, bias=True,
             weighted=False, pad_rows=3, seed=1)
    c.run(dg)
    c.check()


@pytest.mark.parametrize("fmt", FORMATS)
def test_dropped_and_repeated_choices(dg, fmt):
    ids = [[-1, -1, -1], [0, 0, 0], [2, -7, 2], [3, 1, 4], [100, 2, -1], [1, 3, 0]]
    c = Case(fmt, 6, 3, 4, 128, 96, 64, "f16", ids=ids, bias=True, seed=2)
    c.run(dg)
    c.check()
    assert (c.d[0] == 0).all()
    # one token that names one expert more often than a unit has slots
    one = Case(fmt, 1, 12, 4, 128, 96, 64, "f16", ids=[[1] * 11 + [3]], seed=3)
    one.run(dg)
    one.check()
    none = Case(fmt, 2, 2, 4, 128, 96, 64, "f16", ids=[[-1, 9], [4, -2]], seed=4)
    none.run(dg)
    none.check()
    assert (none.d == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_slots_of_one_expert(dg, fmt):
    ids = np.zeros((20, 2), np.int32)
    ids[:, 1] = np.arange(20) % 3
    c = Case(fmt, 20, 2, 3, 264, 128, 128, "bf16", True, ids=ids, seed=5)
    c.run(dg)
    c.check()


@pytest.mark.parametrize("fmt", FORMATS)
def test_largest_routing(dg, fmt):
    # 512 slots, 1024 experts
    rng = np.random.default_rng(6)
    ids = rng.integers(0, 1024, (32, 16))
    ids[rng.random(ids.shape) < 0.1] = -1
    c = Case(fmt, 32, 16, 1024, 64, 32, 32, "bf16", ids=ids, seed=6)
    c.run(dg)
    c.check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_special_values(dg, fmt, dtype):
    c = Case(fmt, 6, 2, 4, 200, 64, 80, dtype, seed=7)
    x = c.x64.copy()
    x[0, 3], x[1, 199], x[2, 100] = np.inf, np.nan, -np.inf
    x[3] = 0.0
    x[4] = 0.0
    x[4, 7] = 2.0 ** -24   # a lone tiny value
    x[5, 0] = 6e4          # the others far below it
    c.x.copy_(torch.from_numpy(x).to(c.x.dtype))
    c.x64 = c.x.double().cpu().numpy()
    c.run(dg)
    d = c.d.double().cpu().numpy()
    assert not np.isfinite(d[:3]).any() and np.isnan(d[1]).all()
    with np.errstate(invalid="ignore"):
        y, bound = c.wanted()
    assert (np.abs(d - y) <= bound)[3:].all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale", [2.0 ** -30, 2.0 ** 20])
def test_range_of_the_hidden_values(dg, fmt, scale):
    # the range of FP32 in between, beyond that of 16 bits
    c = Case(fmt, 3, 2, 4, 256, 128, 64, "bf16", seed=8)
    of = -1 if fmt == "nvf4" else 1
    c.up[of].mul_(scale)
    c.up64 = c.up64 * scale
    c.down[of].mul_(1 / scale)
    c.down64 = c.down64 / scale
    c.run(dg)
    c.check()


@pytest.mark.parametrize("fmt", FORMATS)
def test_scratch_is_left_alone_past_its_size(dg, fmt):
    c = Case(fmt, 3, 2, 4, 256, 136, 72, "f16", seed=9)
    need = dg.lib().dg_moe_layer_scratch(3, 2, 136, 72)
    room = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN wherever unwritten
    keep = dg._scratch
    dg._scratch = lambda torch, n, device, stream: room
    try:
        c.run(dg, stream=torch.cuda.current_stream())
    finally:
        dg._scratch = keep
    dg.check_status()
    c.check()
    assert (room[need:] == 0xFF).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_graphs_and_streams(dg, fmt):
    """Two captured layers, each with scratch of its own, replayed at once on new values."""
    runs = []
    for seed in (10, 11):
        c = Case(fmt, 4, 2, 8, 512, 256, 512, "bf16", True, seed=seed)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            c.run(dg)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for _ in range(3):
                c.run(dg)
        runs.append((c, s, graph))
    for c, _, _ in runs:
        rng = np.random.default_rng(12)
        c.ids64 = rng.integers(-1, 8, c.ids64.shape).astype(np.int32)
        c.ids.copy_(gpu(c.ids64))
        c.x.copy_(c.x * 1.5)
        c.x64 = c.x.double().cpu().numpy()
        c.d.zero_()
    torch.cuda.synchronize()
    for _, s, graph in runs:
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    for c, _, _ in runs:
        c.check()
    c = runs[0][0]
    for stream in (runs[1][1], runs[1][1].cuda_stream, 0):
        c.d.zero_()
        torch.cuda.synchronize()
        c.run(dg, stream=stream)
        torch.cuda.synchronize()
        c.check()


@pytest.mark.parametrize("fmt", FORMATS)
def test_inputs_written_just_before(dg, fmt):
    """Choices, tokens and weights that kernels on the same stream have just written: nothing is
    read before they are done."""
    c = Case(fmt, 2, 2, 4, 512, 1024, 512, "bf16", seed=13)
    c.run(dg)
    want = c.d.clone()
    x, ids, codes = c.x.clone(), c.ids.clone(), [c.up[0].clone(), c.down[0].clone()]
    big = torch.randn(6000, 6000, device="cuda")
    for _ in range(5):
        c.ids.fill_(3)
        c.x.zero_()
        for w in (c.up[0], c.down[0]):
            w.view(torch.uint8).zero_()
        torch.cuda.synchronize()
        big @ big  # keeps the GPU busy while the rest is queued
        c.ids.copy_(ids)
        c.x.copy_(x)
        c.up[0].view(torch.uint8).copy_(codes[0].view(torch.uint8))
        c.down[0].view(torch.uint8).copy_(codes[1].view(torch.uint8))
        c.run(dg)
        assert torch.equal(c.d, want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_largest_tokens_by_width(dg, fmt):
    # as many tokens of a width as shared memory takes, and one more
    width = 2048
    fits = max(t for t in range(1, 64) if t * (2 * width + 64) + 12 * (t + 4) + 28 * t <= 150 * 1024 - 32)
    c = Case(fmt, fits, 1, 4, width, 64, 40, "bf16", seed=14)
    c.run(dg)
    c.check()
    more = Case(fmt, fits + 2, 1, 4, width, 64, 40, "bf16", seed=14)
    with pytest.raises(dg.DgError, match="shared memory"):
        more.run(dg)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens,top_k,count,width,hidden,out,dtype,gated", [
    (5, 2, 3, 8500, 128, 48, "bf16", True),
    (1, 2, 3, 17000, 40, 24, "f16", False),
    (2, 2, 3, 64, 17000, 40, "bf16", False),
    (9, 1, 2, 72, 16900, 33, "f16", False),
])
def test_long_rows(dg, fmt, tokens, top_k, count, width, hidden, out, dtype, gated):
    # more stages of K than a lane each holds the weight scales of
    c = Case(fmt, tokens, top_k, count, width, hidden, out, dtype, gated, seed=hidden)
    c.run(dg)
    dg.check_status()
    c.check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens,top_k", [(1, 512), (240, 2), (33, 1), (16, 2), (11, 3), (170, 3)])
def test_slots(dg, fmt, tokens, top_k):
    # up to 32 slots and more, of one expert and of many
    rng = np.random.default_rng(tokens)
    for count in (1, 3, 40):
        ids = rng.integers(-1 if count > 1 else 0, count, (tokens, top_k))
        c = Case(fmt, tokens, top_k, count, 40, 64, 24, "f16", ids=ids, seed=count)
        c.run(dg)
        c.check()
    dg.check_status()
