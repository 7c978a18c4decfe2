"""The expert layer behind kernels of this library that let the next kernel start as soon as
they have started themselves, and then write what the layer reads: tokens, or the weights of
either product, which the layer's second kernel reads before its own wait; and a layer whose
tokens are another's results."""

import numpy as np
import pytest
import torch

from test_gpu_moe_layer import dg  # noqa: F401

pytestmark = pytest.mark.gpu

TOKENS, TOP_K, COUNT, WIDTH, HIDDEN = 4, 4, 32, 2048, 2048


class Inputs:
    """Where the layer reads from, zeroed by stale(), and steps that write it: the tokens are
    the last rows of a large matrix that is read back from 4 bits."""

    def __init__(self, dg, fmt, seed):  # noqa: F811
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda").bfloat16()
        self.dg, self.fmt = dg, fmt
        self.ids = torch.stack([torch.randperm(COUNT, generator=g, device="cuda")[:TOP_K]
                                for _ in range(TOKENS)]).int()
        self.weights = torch.rand(TOKENS, TOP_K, generator=g, device="cuda")
        self.rows = normal(8192, WIDTH)
        self.rows4 = dg.quantize_nvf4(self.rows)
        self.x = self.rows[-TOKENS:]
        self.w = [normal(COUNT, HIDDEN, WIDTH) / 45, normal(COUNT, WIDTH, HIDDEN) / 45]
        if fmt == "nvf4":
            self.q = [dg.nvf4_buffers(*w.shape) for w in self.w]
        else:
            self.q = [(torch.empty(w.shape, dtype=torch.float8_e4m3fn, device="cuda"),
                       torch.empty(COUNT, w.shape[1] // 128, w.shape[2] // 128, device="cuda"))
                      for w in self.w]
        self.d = torch.empty(TOKENS, WIDTH, dtype=torch.bfloat16, device="cuda")
        self.d2 = torch.empty_like(self.d)

    def stale(self):
        self.rows.zero_()
        for t in self.q[0] + self.q[1] + (self.d, self.d2):
            t.view(torch.uint8).zero_()
        torch.cuda.synchronize()

    def write(self, what):
        if what == "x":
            return self.dg.dequantize_nvf4(*self.rows4, self.rows)
        i = ("up", "down").index(what)
        if self.fmt == "nvf4":
            return self.dg.quantize_nvf4(self.w[i], out=self.q[i])
        for e in range(COUNT):
            self.dg.quantize_fp8(self.w[i][e], block_rows=128,
                                 out=(self.q[i][0][e], self.q[i][1][e]))

    def run(self, order):
        for what in order:
            self.write(what)
        self.dg.moe_layer(self.x, self.ids, self.weights, *self.q, self.d)
        self.dg.moe_layer(self.d, self.ids, self.weights, *self.q, self.d2)

    def results(self):
        torch.cuda.synchronize()
        return self.d.clone(), self.d2.clone()


@pytest.mark.parametrize("fmt", ["fp8", "nvf4"])
@pytest.mark.parametrize("order", [("up", "down", "x"), ("down", "x", "up"), ("x", "up", "down")])
def test_layer_behind_its_inputs_writers(dg, fmt, order):  # noqa: F811
    c = Inputs(dg, fmt, 1)
    for what in order:
        c.write(what)
        torch.cuda.synchronize()
    dg.moe_layer(c.x, c.ids, c.weights, *c.q, c.d)
    torch.cuda.synchronize()
    dg.moe_layer(c.d, c.ids, c.weights, *c.q, c.d2)
    want = c.results()
    assert all((t != 0).any() and torch.isfinite(t).all() for t in want)
    for _ in range(4):
        c.stale()
        c.run(order)
        assert all(torch.equal(a, b) for a, b in zip(c.results(), want))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c.run(order)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.run(order)
    for _ in range(4):
        c.stale()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(c.results(), want))
    dg.check_status()


def test_many_layers_in_a_row(dg):  # noqa: F811
    """Each layer's tokens are the results of the one before, with no other kernel between."""
    c = Inputs(dg, "nvf4", 2)
    for what in ("x", "up", "down"):
        c.write(what)
    t = [c.x.clone()] + [torch.empty_like(c.d) for _ in range(12)]

    def step(sync):
        for a, b in zip(t, t[1:]):
            dg.moe_layer(a, c.ids, c.weights, *c.q, b)
            if sync:
                torch.cuda.synchronize()
    step(True)
    want = [v.clone() for v in t]
    assert np.isfinite([float(v.float().norm()) for v in want]).all()
    for _ in range(3):
        for v in t[1:]:
            v.zero_()
        torch.cuda.synchronize()
        step(False)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(t, want))
